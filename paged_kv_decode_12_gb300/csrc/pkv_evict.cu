// pkv_evict.cu -- a cache cut to a budget of tokens per KV head by the weights it has
// gathered.
//
// For every sequence b of length L > keep and KV head g: the first `sinks` tokens and the
// last `recent` stay; of the others the keep - sinks - recent with the largest
// acc[b][g][t] stay (of equal ones the lowest t; NaN counts as the least).  Each head
// keeps a set of its own -- a page holds its heads' rows apart -- and keys are stored
// rotated, so a row keeps its position's rotation wherever it lies.  The kept rows are
// copied bit by bit, in order, to slots 0 .. keep-1 of the destination pages; acc is
// compacted the same way.  A sequence with L <= keep is copied whole.
//
// Two launches.  select_kernel: one CTA per (sequence, KV head) finds the value of the
// smallest kept weight by a radix selection (8 bits a pass over order-preserving 32-bit
// keys, counts in shared memory), then writes the kept indices in order with one ranked
// pass.  copy_kernel: one CTA per (sequence, destination page), every row of the page's
// eight heads gathered by 16-byte moves.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"

namespace pkv {
namespace {

using namespace dev;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 256;

// Ascending unsigned order = ascending float order; both zeros are one value, NaN is least.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (x != x)
        return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ bool evict_length_ok(int L, int src_blocks, int dst_blocks, int keep)
{
    return L >= 0 && L <= src_blocks * kPage && min(L, keep) <= dst_blocks * kPage;
}

__global__ void __launch_bounds__(kSelThreads)
select_kernel(const int32_t *__restrict__ seq_lens, int src_blocks, int dst_blocks, int keep, int recent, int sinks,
              const float *acc, int64_t acc_stride, float *acc_out, int64_t acc_out_stride, int32_t *__restrict__ kept,
              int32_t *__restrict__ err)
{
    __shared__ int hist[kBins];
    __shared__ int warp_sum[kSelWarps];
    __shared__ int pick[2];
    const int g = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    allow_dependent_launch();
    const size_t row = (size_t)b * kHkv + g;
    const float *w = acc + row * acc_stride;
    float *w_out = acc_out + row * acc_out_stride;
    int32_t *k_out = kept + row * keep;
    int L = seq_lens[b];
    if (!evict_length_ok(L, src_blocks, dst_blocks, keep)) {
        if (tid == 0 && g == 0 && err)
            atomicOr(err, PKV_DEVERR_LENGTH);
        L = 0;
    }
    const int n = min(L, keep);
    // of the tokens lo .. hi-1 the `need` heaviest stay; all others stay
    const int lo = L > keep ? sinks : L, hi = L > keep ? L - recent : L;
    const int need = L > keep ? keep - sinks - recent : 0;
    uint32_t bar = 0;  // the key of the least token kept, and how many of that key are kept
    int ties = 0;
    if (need > 0) {
        int left = need;
        for (int shift = 24; shift >= 0; shift -= 8) {
            const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
            for (int i = tid; i < kBins; i += kSelThreads)
                hist[i] = 0;
            __syncthreads();
            for (int t = lo + tid; t < hi; t += kSelThreads) {
                const uint32_t k = order_key(w[t]);
                if ((k & mask) == bar)
                    atomicAdd(&hist[(k >> shift) & (kBins - 1)], 1);
            }
            __syncthreads();
            if (warp == 0) {  // the bin, from the top, in which the left-th key lies
                int c[kBins / 32], sum = 0;
#pragma unroll
                for (int i = 0; i < kBins / 32; ++i) {
                    c[i] = hist[kBins - 1 - (lane * (kBins / 32) + i)];
                    sum += c[i];
                }
                int x = sum;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(kFull, x, off);
                    if (lane >= off)
                        x += y;
                }
                int above = x - sum;
#pragma unroll
                for (int i = 0; i < kBins / 32; ++i) {
                    if (above < left && left <= above + c[i]) {
                        pick[0] = kBins - 1 - (lane * (kBins / 32) + i);
                        pick[1] = left - above;
                    }
                    above += c[i];
                }
            }
            __syncthreads();
            bar |= (uint32_t)pick[0] << shift;
            left = pick[1];
            __syncthreads();
        }
        ties = left;
    }
    // the kept tokens in order: ranks within tiles of kSelThreads tokens
    int done = 0, tied = 0;
    for (int t0 = 0; t0 < L; t0 += kSelThreads) {
        const int t = t0 + tid;
        const float x = t < L ? w[t] : 0.f;
        const bool middle = t >= lo && t < hi;
        const uint32_t k = middle ? order_key(x) : 0u;
        const bool tie = middle && need > 0 && k == bar;
        const bool sure = t < L && (!middle || (need > 0 && k > bar));
        // (ties, sure ones) before this token, packed in one word: tiles have 1024 tokens
        const uint32_t bt_ = __ballot_sync(kFull, tie), bs = __ballot_sync(kFull, sure);
        if (lane == 0)
            warp_sum[warp] = __popc(bt_) << 16 | __popc(bs);
        __syncthreads();
        int before = 0, total = 0;
#pragma unroll
        for (int i = 0; i < kSelWarps; ++i) {
            const int v = warp_sum[i];
            before += i < warp ? v : 0;
            total += v;
        }
        const uint32_t lower = (1u << lane) - 1;
        const int ties_before = tied + (before >> 16) + __popc(bt_ & lower);
        const int sure_before = (before & 0xffff) + __popc(bs & lower);
        const int taken_before = min(ties_before, ties) - min(tied, ties);
        const bool keep_it = sure || (tie && ties_before < ties);
        if (keep_it) {
            const int i = done + sure_before + taken_before;
            k_out[i] = t;
            w_out[i] = x;
        }
        const int tied_now = tied + (total >> 16);
        done += (total & 0xffff) + min(tied_now, ties) - min(tied, ties);
        tied = tied_now;
        __syncthreads();
    }
    for (int i = n + tid; i < keep; i += kSelThreads)
        k_out[i] = -1;
    for (int64_t i = n + tid; i < acc_out_stride; i += kSelThreads)
        w_out[i] = 0.f;
}

constexpr int kCopyThreads = 256;

// 16 bytes of a BF16 page: row r of the page's 2 x 8 x 16 rows, part c of 8.
__global__ void __launch_bounds__(kCopyThreads)
copy_bf16_kernel(char *slab, int num_pages, const int32_t *__restrict__ seq_lens, const int32_t *__restrict__ bt_src,
                 int src_blocks, const int32_t *__restrict__ bt_dst, int dst_blocks, int keep,
                 const int32_t *__restrict__ kept, int32_t *lens_out, int32_t *__restrict__ err)
{
    const int j = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    grid_dependency_wait();
    allow_dependent_launch();
    const int L = seq_lens[b];
    const bool ok = evict_length_ok(L, src_blocks, dst_blocks, keep);
    const int n = ok ? min(L, keep) : 0;
    if (j == 0 && tid == 0)
        lens_out[b] = n;
    if (j * kPage >= n)
        return;
    const int dst = bt_dst[(size_t)b * dst_blocks + j];
    if (dst < 0 || dst >= num_pages) {
        if (tid == 0 && err)
            atomicOr(err, PKV_DEVERR_PAGE_RANGE);
        return;
    }
    const int slot = (tid >> 3) & 15, part = tid & 7, kv = tid >> 7;  // 2 x 16 rows x 8 parts
    const int i = j * kPage + slot;
    if (i >= n)
        return;
#pragma unroll
    for (int g = 0; g < kHkv; ++g) {
        const int t = kept[((size_t)b * kHkv + g) * keep + i];
        const int src = bt_src[(size_t)b * src_blocks + t / kPage];
        if (src < 0 || src >= num_pages) {
            if (err)
                atomicOr(err, PKV_DEVERR_PAGE_RANGE);
            continue;
        }
        const size_t at = ((size_t)(kv * kHkv + g) * kPage) * kD * 2 + part * 16;
        *reinterpret_cast<uint4 *>(slab + (size_t)dst * PKV_PAGE_BYTES + at + slot * kD * 2) =
            *reinterpret_cast<const uint4 *>(slab + (size_t)src * PKV_PAGE_BYTES + at + (t % kPage) * kD * 2);
    }
}

// The bytes of parity `odd` of a 16-byte chunk of V codes, as 8 bytes.
__device__ __forceinline__ uint2 parity_bytes(uint4 x, int odd)
{
    const uint32_t sel = odd ? 0x7531u : 0x6420u;
    return make_uint2(__byte_perm(x.x, x.y, sel), __byte_perm(x.z, x.w, sel));
}

// FP8 pages: warp = KV head.  K codes: 16 rows x 4 parts of 16 bytes; V codes: 8 token
// pairs x 8 chunks of 16 bytes, a chunk's two tokens gathered from their own lines;
// scales: 2 x 16.
__global__ void __launch_bounds__(kCopyThreads)
copy_fp8_kernel(char *slab, int num_pages, const int32_t *__restrict__ seq_lens, const int32_t *__restrict__ bt_src,
                int src_blocks, const int32_t *__restrict__ bt_dst, int dst_blocks, int keep,
                const int32_t *__restrict__ kept, int32_t *lens_out, int32_t *__restrict__ err)
{
    const int j = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, g = tid >> 5, lane = tid & 31;
    grid_dependency_wait();
    allow_dependent_launch();
    const int L = seq_lens[b];
    const bool ok = evict_length_ok(L, src_blocks, dst_blocks, keep);
    const int n = ok ? min(L, keep) : 0;
    if (j == 0 && tid == 0)
        lens_out[b] = n;
    if (j * kPage >= n)
        return;
    const int dst = bt_dst[(size_t)b * dst_blocks + j];
    if (dst < 0 || dst >= num_pages) {
        if (tid == 0 && err)
            atomicOr(err, PKV_DEVERR_PAGE_RANGE);
        return;
    }
    // lanes 0..15 hold the page's 16 tokens: source slot and the unit's address (-1: none)
    int64_t unit = -1;
    int slot = 0;
    const int m = min(kPage, n - j * kPage);
    if (lane < m) {
        const int t = kept[((size_t)b * kHkv + g) * keep + j * kPage + lane];
        const int src = bt_src[(size_t)b * src_blocks + t / kPage];
        if (src >= 0 && src < num_pages) {
            unit = (int64_t)src * kFp8PageBytes + g * kFp8Unit;
            slot = t % kPage;
        } else if (err) {
            atomicOr(err, PKV_DEVERR_PAGE_RANGE);
        }
    }
    char *to = slab + (size_t)dst * kFp8PageBytes + g * kFp8Unit;
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // K codes
        const int s = i * 8 + (lane >> 2), part = lane & 3;
        const int64_t u = __shfl_sync(kFull, unit, s);
        const int from = __shfl_sync(kFull, slot, s);
        if (u >= 0)
            *reinterpret_cast<uint4 *>(to + s * kD + part * 16) =
                *reinterpret_cast<const uint4 *>(slab + u + from * kD + part * 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // V codes: pair p, dims 8c .. 8c+7
        const int p = i * 4 + (lane >> 3), c = lane & 7;
        const int64_t u0 = __shfl_sync(kFull, unit, 2 * p), u1 = __shfl_sync(kFull, unit, 2 * p + 1);
        const int s0 = __shfl_sync(kFull, slot, 2 * p), s1 = __shfl_sync(kFull, slot, 2 * p + 1);
        const auto chunk = [&](int s) { return fp8::kFp8Tile + (fp8::v_code_offset(s, 8 * c) & ~15); };
        uint4 *out = reinterpret_cast<uint4 *>(to + chunk(2 * p));
        if (u0 < 0 && u1 < 0)
            continue;
        // a slot without a token keeps its bytes
        const uint4 old = (u0 < 0 || u1 < 0) ? *out : make_uint4(0, 0, 0, 0);
        const uint2 e = u0 >= 0 ? parity_bytes(*reinterpret_cast<const uint4 *>(slab + u0 + chunk(s0)), s0 & 1)
                                : parity_bytes(old, 0);
        const uint2 o = u1 >= 0 ? parity_bytes(*reinterpret_cast<const uint4 *>(slab + u1 + chunk(s1)), s1 & 1)
                                : parity_bytes(old, 1);
        *out = make_uint4(__byte_perm(e.x, o.x, 0x5140), __byte_perm(e.x, o.x, 0x7362),
                          __byte_perm(e.y, o.y, 0x5140), __byte_perm(e.y, o.y, 0x7362));
    }
    {  // scales: K rows' then V rows'
        const int s = lane & 15, kv = lane >> 4;
        const int64_t u = __shfl_sync(kFull, unit, s);
        const int from = __shfl_sync(kFull, slot, s);
        if (u >= 0)
            reinterpret_cast<float *>(to + kFp8UnitCodes)[kv * kPage + s] =
                reinterpret_cast<const float *>(slab + u + kFp8UnitCodes)[kv * kPage + from];
    }
}

bool evict_args_ok(int B, int keep)
{
    return B >= 1 && B <= 65535 && keep >= 1 && keep <= (1 << 20) * kPage;
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_evict_workspace_bytes(int B, int keep)
{
    using namespace pkv;
    if (!evict_args_ok(B, keep))
        return 0;
    return (size_t)B * kHkv * keep * sizeof(int32_t);
}

extern "C" int pkv_evict(const pkv_pool *pool, const int32_t *bt_src_dev, int src_blocks, const int32_t *seq_lens_dev,
                         int B, const int32_t *bt_dst_dev, int dst_blocks, int keep, int recent, int sinks,
                         const float *acc, int64_t acc_stride, float *acc_out, int64_t acc_out_stride, int32_t *kept,
                         int32_t *seq_lens_out, void *workspace, size_t workspace_bytes, int32_t *dev_err_flag,
                         void *cuda_stream)
{
    using namespace pkv;
    if (!pool || !bt_src_dev || !seq_lens_dev || !bt_dst_dev || !acc || !acc_out || !seq_lens_out ||
        !evict_args_ok(B, keep))
        return PKV_ERR_INVALID_ARG;
    if (src_blocks < 1 || src_blocks > (1 << 20) || dst_blocks < 1 || dst_blocks > (1 << 20) || recent < 0 || sinks < 0 ||
        (int64_t)recent + sinks > keep)
        return PKV_ERR_INVALID_ARG;
    if (acc_stride < (int64_t)src_blocks * kPage || acc_out_stride < (int64_t)dst_blocks * kPage ||
        (acc == acc_out && acc_stride != acc_out_stride))
        return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(acc) | reinterpret_cast<uintptr_t>(acc_out)) & 3u)
        return PKV_ERR_INVALID_ARG;
    if (!kept) {
        if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 3u))
            return PKV_ERR_INVALID_ARG;
        if (workspace_bytes < pkv_evict_workspace_bytes(B, keep))
            return PKV_ERR_WORKSPACE_TOO_SMALL;
        kept = static_cast<int32_t *>(workspace);
    }
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    // rows written here are read by later launches: the next decode launch on the pool may
    // not copy pages before its dependency wait
    pool->serialize_next_launch = true;
    if (const int st = launch_kernel(select_kernel, dim3(kHkv, B), dim3(kSelThreads), 0, s, false, seq_lens_dev, src_blocks,
                                     dst_blocks, keep, recent, sinks, acc, acc_stride, acc_out, acc_out_stride, kept,
                                     dev_err_flag);
        st != PKV_OK)
        return st;
    const int pages = std::min(dst_blocks, (keep + kPage - 1) / kPage);
    auto kernel = pool->kv_format == PKV_KV_FP8 ? copy_fp8_kernel : copy_bf16_kernel;
    return launch_kernel(kernel, dim3(pages, B), dim3(kCopyThreads), 0, s, true, pool->slab, pool->num_pages,
                         seq_lens_dev, bt_src_dev, src_blocks, bt_dst_dev, dst_blocks, keep,
                         static_cast<const int32_t *>(kept), seq_lens_out, dev_err_flag);
}
