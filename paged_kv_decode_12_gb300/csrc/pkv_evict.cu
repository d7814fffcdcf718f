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
// by histograms of order-preserving 32-bit keys, then writes the kept indices
// in order with one ranked pass.  copy_*_kernel: a warp per (sequence, KV head, run of
// destination pages) gathers the rows by 16-byte moves.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"

namespace pkv {
namespace {

using namespace dev;

// Ascending unsigned order = ascending float order; both zeros are one value, NaN is least.
// No float has the keys kNone (no token) and kStays (a token that is not up for choice).
constexpr uint32_t kNone = 0u, kNan = 1u, kStays = 0xffffffffu;

__device__ __forceinline__ uint32_t order_key(float x)
{
    if (x != x)
        return kNan;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ bool evict_length_ok(int L, int src_blocks, int dst_blocks, int keep)
{
    return L >= 0 && L <= src_blocks * kPage && min(L, keep) <= dst_blocks * kPage;
}

constexpr int kBins = 1024;

// One CTA of WARPS warps per (sequence, KV head); warp v has the row's tokens 32 v per .. and on,
// `per` times 32 of them.  PER > 0: their keys (at most PER a thread) stay in registers; PER = 0,
// for rows longer than that: they are read again in every step.
//
// The least kept key is found by histograms: the keys up for choice in a range (at first from their
// least to their greatest) fall into up to 1024 bins of equal width, the bin that holds the wanted
// rank becomes the next range, and a range of one key, or one that is kept whole, ends the search:
// four steps at most, two as a rule.  Once no more keys than threads are left, they are gathered,
// one a thread, for the steps left.  The kept tokens' ranks then take one more barrier: every warp
// counts its own first.  What bounds it is the number of instructions and barriers, so few warps
// with many keys each (512 rows of 6000 weights: 62 us with 32 warps of 8 keys that counted bit by
// bit, 29 us with 8 warps of 32, 23 us by histograms).
template <int WARPS, int PER>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 4 : 1)
select_kernel(const int32_t *__restrict__ seq_lens, int src_blocks, int dst_blocks, int keep, int recent, int sinks,
              const float *acc, int64_t acc_stride, float *acc_out, int64_t acc_out_stride, int32_t *__restrict__ kept,
              int32_t *__restrict__ err)
{
    constexpr int kThreadsHere = WARPS * 32;
    constexpr int kPerThread = kBins / kThreadsHere;  // bins a thread
    __shared__ int sums[32], tie_sums[32], gathered, bins[kBins];
    __shared__ uint32_t few[kThreadsHere], least[32], greatest[32];
    __shared__ int3 found;
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
    const int per = (L + kThreadsHere - 1) / kThreadsHere, t0 = warp * per * 32 + lane;
    // every weight is read, whether it matters or not, so that a thread's reads are in flight at once
    const auto weight = [&](int i) { return w[max(min(t0 + i * 32, L - 1), 0)]; };
    const auto key = [&](int i, float x) {
        const int t = t0 + i * 32;
        return i >= per || t >= L ? kNone : L <= keep || t < sinks || t >= L - recent ? kStays : order_key(x);
    };
    uint32_t held[PER > 0 ? PER : 1];
    if constexpr (PER > 0) {
#pragma unroll
        for (int i0 = 0; i0 < PER; i0 += 8) {
#pragma unroll
            for (int i = i0; i < i0 + 8; ++i)
                held[i] = i0 < per ? __float_as_uint(weight(i)) : 0u;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            held[i] = key(i, __uint_as_float(held[i]));
    }
    // f(i, key) of this thread's tokens (and of some behind them, eight to a branch)
    const auto each = [&](const auto &f) {
        if constexpr (PER > 0) {
#pragma unroll
            for (int i0 = 0; i0 < PER; i0 += 8)
                if (i0 < per)
#pragma unroll
                    for (int i = i0; i < i0 + 8; ++i)
                        f(i, held[i]);
        } else {
#pragma unroll 4
            for (int i = 0; i < per; ++i)
                f(i, key(i, weight(i)));
        }
    };
    // kept: keys above `bar`, and the first `ties` tokens of that key
    uint32_t bar = kNone;
    int ties = 0;
    int want = keep - sinks - recent;  // of the keys up for choice that are left, how many are kept
    if (L > keep && want == 0) {
        bar = kStays - 1;
    } else if (L > keep) {
        uint32_t lo = kStays, hi = kNone;
        each([&](int, uint32_t k) {
            if (k != kNone && k != kStays) {
                lo = min(lo, k);
                hi = max(hi, k);
            }
        });
        lo = __reduce_min_sync(kFull, lo);
        hi = __reduce_max_sync(kFull, hi);
        if (lane == 0) {
            least[warp] = lo;
            greatest[warp] = hi;
        }
        __syncthreads();
        lo = __reduce_min_sync(kFull, lane < WARPS ? least[lane] : kStays);
        hi = __reduce_max_sync(kFull, lane < WARPS ? greatest[lane] : kNone);
        int left = L - sinks - recent;  // keys in lo .. hi; more than `want`, and `want` is positive
        const auto narrow = [&](const auto &each_key) {
            const int shift = max(22 - __clz(hi - lo), 0);  // hi - lo in ten bits
#pragma unroll
            for (int i = 0; i < kPerThread; ++i)
                bins[tid * kPerThread + i] = 0;
            __syncthreads();
            each_key([&](int, uint32_t k) {
                if (k - lo <= hi - lo)
                    atomicAdd(&bins[(k - lo) >> shift], 1);
            });
            __syncthreads();
            int own[kPerThread], from = 0;  // this thread's bins; keys in them and in all above them
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) {
                own[i] = bins[tid * kPerThread + i];
                from += own[i];
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_down_sync(kFull, from, off);
                if (lane + off < 32)
                    from += y;
            }
            if (lane == 0)
                sums[warp] = from;
            __syncthreads();
            from += __reduce_add_sync(kFull, lane > warp && lane < WARPS ? sums[lane] : 0);
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) {
                if (from >= want && from - own[i] < want)
                    found = make_int3(tid * kPerThread + i, from - own[i], own[i]);
                from -= own[i];
            }
            __syncthreads();
            lo += (uint32_t)found.x << shift;
            hi = min(hi, lo + ((1u << shift) - 1));
            want -= found.y;
            left = found.z;
        };
        while (lo != hi && left != want && left > kThreadsHere)
            narrow(each);
        if (lo != hi && left != want) {
            if (tid == 0)
                gathered = 0;
            __syncthreads();
            each([&](int, uint32_t k) {
                if (k - lo <= hi - lo)
                    few[atomicAdd(&gathered, 1)] = k;
            });
            __syncthreads();
            const uint32_t mine = tid < gathered ? few[tid] : kNone;
            while (lo != hi && left != want)
                narrow([&](const auto &f) { f(0, mine); });
        }
        bar = left == want ? lo - 1 : lo;  // (a range that is kept whole, or one key)
        ties = left == want ? 0 : want;
        __syncthreads();
    }
    int sure = 0, tied = 0;  // of this thread, then of the warps before
    each([&](int, uint32_t k) {
        sure += k > bar;
        tied += k == bar;
    });
    sure = __reduce_add_sync(kFull, sure);
    tied = __reduce_add_sync(kFull, tied);
    if (lane == 0) {
        sums[warp] = sure;
        tie_sums[warp] = tied;
    }
    __syncthreads();
    sure = __reduce_add_sync(kFull, lane < warp ? sums[lane] : 0);
    tied = __reduce_add_sync(kFull, lane < warp ? tie_sums[lane] : 0);
    const uint32_t lower = (1u << lane) - 1;
    each([&](int i, uint32_t k) {
        const bool s = k > bar, e = k == bar;
        const uint32_t bs = __ballot_sync(kFull, s), be = __ballot_sync(kFull, e);
        const int before = tied + __popc(be & lower);  // ties before this token
        if (s || (e && before < ties))
            k_out[sure + __popc(bs & lower) + min(before, ties)] = t0 + i * 32;
        sure += __popc(bs);
        tied += __popc(be);
    });
    __syncthreads();
    // the kept weights, four a thread at a time: all of them are read before any is written, and
    // none comes from further forward than it goes to, so this may be done in place
    constexpr int kRound = 4 * WARPS * 32;
    for (int i0 = 0; i0 < n; i0 += kRound) {
        float x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = i0 + q * WARPS * 32 + tid;
            x[q] = i < n ? w[k_out[i]] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = i0 + q * WARPS * 32 + tid;
            if (i < n)
                w_out[i] = x[q];
        }
    }
    __syncthreads();
    for (int i = n + tid; i < keep; i += WARPS * 32)
        k_out[i] = -1;
    for (int64_t i = n + tid; i < acc_out_stride; i += WARPS * 32)
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
    // rows written here are read by later launches: a decode launch behind them may not copy pages
    // before its dependency wait
    pages_written(pool, s);
    const int longest = src_blocks * kPage, threads = longest <= 8 * 32 * 32 ? 8 * 32 : 32 * 32;
    const auto select = longest <= 8 * 32 * 32    ? select_kernel<8, 32>
                        : longest <= 32 * 32 * 32 ? select_kernel<32, 32>
                                                  : select_kernel<32, 0>;
    if (const int st = launch_kernel(select, dim3(kHkv, B), dim3(threads), 0, s, true, seq_lens_dev, src_blocks,
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
