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
// Two launches.  select_kernel: one CTA per (sequence, KV head) finds the least kept weight
// by its bits, from the top, over order-preserving 32-bit keys, then writes the kept indices
// in order with one ranked pass.  copy_*_kernel: a warp per (sequence, KV head, run of
// destination pages) gathers the rows by 16-byte moves.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"

namespace pkv {
namespace {

using namespace dev;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

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

// The keys of tokens lo .. hi-1 of a row, PER of them a thread in registers (token i * 1024 +
// thread), or, for rows longer than that (PER = 0), read again in every pass.
template <int PER>
struct RowKeys {
    int tiles;
    uint32_t k[PER];
    __device__ __forceinline__ RowKeys(const float *w, int lo, int hi) : tiles((hi + kSelThreads - 1) / kSelThreads)
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = i * kSelThreads + threadIdx.x;
            k[i] = t >= lo && t < hi ? order_key(w[t]) : 0u;
        }
    }
    // how many of this thread's keys are at least each of three values (none of them 0)
    __device__ __forceinline__ void count(const uint32_t (&v)[3], int (&n)[3]) const
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (i >= tiles)
                break;
#pragma unroll
            for (int c = 0; c < 3; ++c)
                n[c] += k[i] >= v[c];
        }
    }
};

template <>
struct RowKeys<0> {
    const float *w;
    int lo, hi;
    __device__ __forceinline__ RowKeys(const float *w_, int lo_, int hi_) : w(w_), lo(lo_), hi(hi_) {}
    __device__ __forceinline__ void count(const uint32_t (&v)[3], int (&n)[3]) const
    {
        for (int t = lo + threadIdx.x; t < hi; t += kSelThreads) {
            const uint32_t k = order_key(w[t]);
#pragma unroll
            for (int c = 0; c < 3; ++c)
                n[c] += k >= v[c];
        }
    }
};

// One CTA per (sequence, KV head).  Two bits of the least kept key at a time, from the top: the
// largest prefix of which at least `need` keys are not below.  Counting keys held in registers
// against three candidates takes no atomics (a histogram's bins would be few and crowded: weights
// share their exponents) and one barrier a step.
template <int PER>
__global__ void __launch_bounds__(kSelThreads, PER > 0 && PER <= 8 ? 2 : 1)
select_kernel(const int32_t *__restrict__ seq_lens, int src_blocks, int dst_blocks, int keep, int recent, int sinks,
              const float *acc, int64_t acc_stride, float *acc_out, int64_t acc_out_stride, int32_t *__restrict__ kept,
              int32_t *__restrict__ err)
{
    __shared__ int sums[2][3][kSelWarps];
    __shared__ int tile_sums[2][kSelWarps];
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
    const RowKeys<PER> keys(w, lo, hi);
    uint32_t bar = 0;     // the key of the least token kept
    int ties = 0;         // how many of that key are kept
    if (need > 0) {
        // keys of NaN are 0 and count like any other: a value of 0 is reached by all hi - lo
        int above = 0;    // keys above every key that begins with bar's bits so far
        for (int shift = 30, step = 0; shift >= 0; shift -= 2, step ^= 1) {
            const uint32_t v[3] = {bar | 1u << shift, bar | 2u << shift, bar | 3u << shift};
            int c[3] = {0, 0, 0};
            keys.count(v, c);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int s = __reduce_add_sync(kFull, c[i]);
                if (lane == 0)
                    sums[step][i][warp] = s;
            }
            __syncthreads();
            int total[3];
#pragma unroll
            for (int i = 0; i < 3; ++i)
                total[i] = __reduce_add_sync(kFull, sums[step][i][lane]);
            // the largest of the four continuations that `need` keys reach
            const int pick = total[2] >= need ? 3 : total[1] >= need ? 2 : total[0] >= need ? 1 : 0;
            if (pick < 3)
                above = total[pick];
            bar |= (uint32_t)pick << shift;
        }
        ties = need - above;
    }
    // the kept tokens in order: ranks within tiles of kSelThreads tokens
    int done = 0, tied = 0;
    for (int i = 0; i * kSelThreads < L; ++i) {
        const int t = i * kSelThreads + tid;
        const float x = t < L ? w[t] : 0.f;
        const bool middle = t >= lo && t < hi;
        const uint32_t k = order_key(x);
        const bool tie = middle && need > 0 && k == bar;
        const bool sure = t < L && (!middle || (need > 0 && k > bar));
        // (ties, sure ones) of each warp, packed in one word: tiles have 1024 tokens
        const uint32_t bt_ = __ballot_sync(kFull, tie), bs = __ballot_sync(kFull, sure);
        if (lane == 0)
            tile_sums[i & 1][warp] = __popc(bt_) << 16 | __popc(bs);
        __syncthreads();
        const int v = tile_sums[i & 1][lane];
        const int total = __reduce_add_sync(kFull, v), before = __reduce_add_sync(kFull, lane < warp ? v : 0);
        const uint32_t lower = (1u << lane) - 1;
        const int ties_before = tied + (before >> 16) + __popc(bt_ & lower);
        const int sure_before = (before & 0xffff) + __popc(bs & lower);
        const int taken_before = min(ties_before, ties) - min(tied, ties);
        if (sure || (tie && ties_before < ties)) {
            const int at = done + sure_before + taken_before;
            k_out[at] = t;
            w_out[at] = x;
        }
        const int tied_now = tied + (total >> 16);
        done += (total & 0xffff) + min(tied_now, ties) - min(tied, ties);
        tied = tied_now;
    }
    __syncthreads();  // with weights in place, the last reads come before the zeros
    for (int i = n + tid; i < keep; i += kSelThreads)
        k_out[i] = -1;
    for (int64_t i = n + tid; i < acc_out_stride; i += kSelThreads)
        w_out[i] = 0.f;
}

constexpr int kCopyThreads = kHkv * 32;  // a warp per KV head

// What both copy kernels' CTAs do: destination tokens 32 * per * blockIdx.x and on of sequence b,
// 32 (two pages) at a time.  A row's address hangs on three loads, each on the one before (kept
// token, table entry, row); the first two are made for the next 32 tokens while these are copied.
struct CopyArgs {
    char *slab;
    int num_pages;
    const int32_t *seq_lens, *bt_src, *bt_dst, *kept;
    int src_blocks, dst_blocks, keep, per;
    int32_t *lens_out, *err;
};

// Lane's source of one destination token.
struct Source {
    int page, slot;  // page -1: none
};

__device__ __forceinline__ Source source_of(const CopyArgs &a, int b, int g, int i, int n)
{
    Source s = {-1, 0};
    if (i < n) {
        const int t = a.kept[((size_t)b * kHkv + g) * a.keep + i];
        s.page = a.bt_src[(size_t)b * a.src_blocks + t / kPage];
        s.slot = t % kPage;
        if (s.page < 0 || s.page >= a.num_pages) {
            s.page = -1;
            if (a.err)
                atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
        }
    }
    return s;
}

template <class CopyPage>
__device__ __forceinline__ void copy_pages(const CopyArgs &a, const CopyPage &copy_page)
{
    const int b = blockIdx.y, g = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int L = a.seq_lens[b];
    grid_dependency_wait();
    allow_dependent_launch();
    const int n = evict_length_ok(L, a.src_blocks, a.dst_blocks, a.keep) ? min(L, a.keep) : 0;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        a.lens_out[b] = n;
    const int first = blockIdx.x * 32 * a.per, end = min(n, first + 32 * a.per);
    if (first >= end)
        return;
    Source s = source_of(a, b, g, first + lane, end);
    for (int i = first; i < end; i += 32) {
        const Source now = s;
        s = source_of(a, b, g, i + 32 + lane, end);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (i + h * kPage >= end)
                break;
            const int dst = a.bt_dst[(size_t)b * a.dst_blocks + i / kPage + h];
            if (dst < 0 || dst >= a.num_pages) {
                if (lane == 0 && a.err)
                    atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
                continue;
            }
            copy_page(dst, g, lane, h * kPage, now);
        }
    }
}

// BF16 pages: 16 K rows and 16 V rows of 128 bytes, 4 rows a load.
__global__ void __launch_bounds__(kCopyThreads) copy_bf16_kernel(CopyArgs a)
{
    copy_pages(a, [&](int dst, int g, int lane, int at, Source s) {
        const size_t head = (size_t)g * kPage * kD * 2 + (lane & 7) * 16;
        uint4 v[2][4];
        int page[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = i * 4 + (lane >> 3);
            page[i] = __shfl_sync(kFull, s.page, at + row);
            const int slot = __shfl_sync(kFull, s.slot, at + row);
            const char *from = a.slab + (size_t)max(page[i], 0) * PKV_PAGE_BYTES + head + slot * kD * 2;
            if (page[i] >= 0) {
                v[0][i] = *reinterpret_cast<const uint4 *>(from);
                v[1][i] = *reinterpret_cast<const uint4 *>(from + PKV_PAGE_BYTES / 2);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = i * 4 + (lane >> 3);
            char *to = a.slab + (size_t)dst * PKV_PAGE_BYTES + head + row * kD * 2;
            if (page[i] >= 0) {
                *reinterpret_cast<uint4 *>(to) = v[0][i];
                *reinterpret_cast<uint4 *>(to + PKV_PAGE_BYTES / 2) = v[1][i];
            }
        }
    });
}

// The bytes of parity `odd` of a 16-byte chunk of V codes, as 8 bytes.
__device__ __forceinline__ uint2 parity_bytes(uint4 x, int odd)
{
    const uint32_t sel = odd ? 0x7531u : 0x6420u;
    return make_uint2(__byte_perm(x.x, x.y, sel), __byte_perm(x.z, x.w, sel));
}

// FP8 pages.  K codes: 16 rows of 4 parts of 16 bytes; V codes: 8 token pairs of 8 chunks of 16
// bytes, a chunk's two tokens gathered from their own lines; row scales: 2 x 16.
__global__ void __launch_bounds__(kCopyThreads) copy_fp8_kernel(CopyArgs a)
{
    copy_pages(a, [&](int dst, int g, int lane, int at, Source s) {
        const auto unit = [&](int page) { return a.slab + (size_t)max(page, 0) * kFp8PageBytes + g * kFp8Unit; };
        const auto chunk = [](int slot, int c) { return fp8::kFp8Tile + (fp8::v_code_offset(slot, 8 * c) & ~15); };
        char *to = unit(dst);
        uint4 k[2], e[2], o[2];
        int kp[2], ep[2], op[2], es[2], os[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = i * 8 + (lane >> 2);
            kp[i] = __shfl_sync(kFull, s.page, at + row);
            const int slot = __shfl_sync(kFull, s.slot, at + row);
            if (kp[i] >= 0)
                k[i] = *reinterpret_cast<const uint4 *>(unit(kp[i]) + slot * kD + (lane & 3) * 16);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // pair p, dims 8c .. 8c+7
            const int p = i * 4 + (lane >> 3), c = lane & 7;
            ep[i] = __shfl_sync(kFull, s.page, at + 2 * p);
            es[i] = __shfl_sync(kFull, s.slot, at + 2 * p);
            op[i] = __shfl_sync(kFull, s.page, at + 2 * p + 1);
            os[i] = __shfl_sync(kFull, s.slot, at + 2 * p + 1);
            // a slot without a token keeps its bytes
            if (ep[i] >= 0)
                e[i] = *reinterpret_cast<const uint4 *>(unit(ep[i]) + chunk(es[i], c));
            if (op[i] >= 0)
                o[i] = *reinterpret_cast<const uint4 *>(unit(op[i]) + chunk(os[i], c));
            if ((ep[i] < 0) != (op[i] < 0)) {
                const uint4 old = *reinterpret_cast<const uint4 *>(to + chunk(2 * p, c));
                if (ep[i] < 0) {
                    e[i] = old;
                    es[i] = 0;
                } else {
                    o[i] = old;
                    os[i] = 1;
                }
            }
        }
        const int sp = __shfl_sync(kFull, s.page, at + (lane & 15)), ss = __shfl_sync(kFull, s.slot, at + (lane & 15));
        const int kv = lane >> 4;
        float f = 0.f;
        if (sp >= 0)
            f = reinterpret_cast<const float *>(unit(sp) + kFp8UnitCodes)[kv * kPage + ss];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (kp[i] >= 0)
                *reinterpret_cast<uint4 *>(to + (i * 8 + (lane >> 2)) * kD + (lane & 3) * 16) = k[i];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int p = i * 4 + (lane >> 3), c = lane & 7;
            if (ep[i] < 0 && op[i] < 0)
                continue;
            const uint2 x = parity_bytes(e[i], es[i] & 1), y = parity_bytes(o[i], os[i] & 1);
            *reinterpret_cast<uint4 *>(to + chunk(2 * p, c)) =
                make_uint4(__byte_perm(x.x, y.x, 0x5140), __byte_perm(x.x, y.x, 0x7362),
                           __byte_perm(x.y, y.y, 0x5140), __byte_perm(x.y, y.y, 0x7362));
        }
        if (sp >= 0)
            reinterpret_cast<float *>(to + kFp8UnitCodes)[kv * kPage + (lane & 15)] = f;
    });
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
    const int longest = src_blocks * kPage;
    const auto select = longest <= 8 * kSelThreads    ? select_kernel<8>
                        : longest <= 32 * kSelThreads ? select_kernel<32>
                                                      : select_kernel<0>;
    if (const int st = launch_kernel(select, dim3(kHkv, B), dim3(kSelThreads), 0, s, true, seq_lens_dev, src_blocks,
                                     dst_blocks, keep, recent, sinks, acc, acc_stride, acc_out, acc_out_stride, kept,
                                     dev_err_flag);
        st != PKV_OK)
        return st;
    // 32 tokens of a head a step; several steps a warp once the GPU is full (8 CTAs on each SM),
    // so that a step's addresses are looked up during the one before
    const int steps = (std::min(dst_blocks * kPage, keep) + 31) / 32;
    CopyArgs c;
    c.slab = pool->slab;
    c.num_pages = pool->num_pages;
    c.seq_lens = seq_lens_dev;
    c.bt_src = bt_src_dev;
    c.bt_dst = bt_dst_dev;
    c.kept = kept;
    c.src_blocks = src_blocks;
    c.dst_blocks = dst_blocks;
    c.keep = keep;
    c.per = (int)std::min<int64_t>(8, ((int64_t)steps * B + 152 * 8 - 1) / (152 * 8));
    c.lens_out = seq_lens_out;
    c.err = dev_err_flag;
    return launch_kernel(pool->kv_format == PKV_KV_FP8 ? copy_fp8_kernel : copy_bf16_kernel,
                         dim3((steps + c.per - 1) / c.per, B), dim3(kCopyThreads), 0, s, true, c);
}
