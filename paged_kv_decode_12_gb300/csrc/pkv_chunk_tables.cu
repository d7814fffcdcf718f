// pkv_chunk_tables.cu -- block tables, positions and slot maps of a step's new tokens, made on the
// GPU from the sequences' lengths.
//
// Sequence b holds len[b] tokens and brings new[b].  With P(n) = ceil(n / 16) it needs
// add[b] = P(len[b] + new[b]) - P(len[b]) pages more in each layer.  The pages come from a list,
// layer by layer and sequence by sequence: with A[b] the sum of add before b, the i-th new page of
// sequence b in layer l is list[used + l * A[B] + A[b] + i].  Token t of the step belongs to the
// sequence b with start[b] <= t < start[b + 1] (start the prefix sums of new), has position
// p = len[b] + t - start[b] and in layer l the slot 16 * table[l][b][p / 16] + p % 16.
//
// The work is two prefix sums over the batch and then stores, 8 bytes a token and layer.  Every CTA
// makes the sums for itself (4096 rows are 8 a thread, and come from L2), so that nothing waits for
// another CTA; the few words that may be the inputs themselves (lengths, the list's count) are
// written by the CTA that draws the last ticket, when all have read them.
//
// What bounds it is latency, one step behind the other (lengths, sums, a search, page ids): 1 token 3.4 us
// and 64 sequences in 16 layers 4.7; 512 sequences, 99456 tokens in 16 layers (14 MB) 9.4 where a copy's
// rate would take 2.1.
#include "pkv_device.cuh"

namespace pkv {
namespace {

using namespace dev;

constexpr int kTablesThreads = 512;
constexpr int kMaxRows = 4096;                       // sequences of a call
constexpr int kRowsPerThread = kMaxRows / kTablesThreads;
constexpr int kTablesCtas = 152;
// Of a token: loads on their way.  (512 sequences: 9.4 us, with 4 of them 9.9, with 16 9.2, but 64 sequences
// 5.0 where 4.7; one load behind each store, which may be to its address for all the compiler knows, 13.4.)
constexpr int kLayersAtOnce = 8;

struct TablesArgs {
    const int32_t *lens, *fresh;
    int B;
    int32_t *bt;
    int max_blocks, layers;
    const int32_t *pages;
    int num_listed;
    const int32_t *used;
    int32_t *used_out;
    int max_tokens;
    int32_t *starts, *lens_out, *pos;
    int64_t *slots;
    int num_pages;
    int *ticket;
    int32_t *err;
    int tile, layer_ctas;  // tokens of a CTA's tile (a power of two), CTAs that share a tile's layers
};

__device__ __forceinline__ int pages_of(int64_t tokens) { return (int)((tokens + kPage - 1) / kPage); }

// The row of a sorted array of prefix sums (n + 1 entries, x below the last) that x falls into.
__device__ __forceinline__ int find_row(const int *sums, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTablesThreads) chunk_tables_kernel(TablesArgs a)
{
    __shared__ int starts[kMaxRows + 1], before[kMaxRows + 1], lens[kMaxRows];
    __shared__ int64_t warp_tokens[kTablesThreads / 32], warp_pages[kTablesThreads / 32];
    grid_dependency_wait();
    allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool reports = blockIdx.x == 0 && blockIdx.y == 0;
    // ---- prefix sums of new tokens and new pages; a row that is not valid brings nothing
    int tokens[kRowsPerThread], add[kRowsPerThread];
    int64_t sum_t = 0, sum_p = 0;
    bool bad_row = false;
    const int per = (a.B + kTablesThreads - 1) / kTablesThreads;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
        tokens[i] = add[i] = 0;
        const int b = threadIdx.x * per + i;
        if (i < per && b < a.B) {
            const int len = a.lens[b], n = a.fresh[b];
            const bool ok = len >= 0 && n >= 0 && (int64_t)len + n <= (int64_t)a.max_blocks * kPage;
            lens[b] = len;
            if (ok) {
                tokens[i] = n;
                add[i] = pages_of((int64_t)len + n) - pages_of(len);
            } else {
                bad_row = true;
            }
            sum_t += tokens[i];
            sum_p += add[i];
        }
    }
    int64_t inc_t = sum_t, inc_p = sum_p;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(kFull, inc_t, off), y = __shfl_up_sync(kFull, inc_p, off);
        if (lane >= off) {
            inc_t += x;
            inc_p += y;
        }
    }
    if (lane == 31) {
        warp_tokens[warp] = inc_t;
        warp_pages[warp] = inc_p;
    }
    bad_row = __syncthreads_or(bad_row);
    int64_t at_t = inc_t - sum_t, at_p = inc_p - sum_p, all_t = 0, all_p = 0;
    for (int w = 0; w < kTablesThreads / 32; ++w) {
        if (w < warp) {
            at_t += warp_tokens[w];
            at_p += warp_pages[w];
        }
        all_t += warp_tokens[w];
        all_p += warp_pages[w];
    }
    // ---- all or nothing
    const int used = *a.used;
    const bool fits = all_t <= a.max_tokens;
    const bool enough = used >= 0 && all_p * a.layers <= (int64_t)a.num_listed - used;
    const bool go = fits && enough;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
        const int b = threadIdx.x * per + i;
        if (i < per && b < a.B) {
            starts[b] = go ? (int)at_t : 0;
            before[b] = go ? (int)at_p : 0;
            at_t += tokens[i];
            at_p += add[i];
        }
    }
    const int T = go ? (int)all_t : 0, total = go ? (int)all_p : 0;
    if (threadIdx.x == 0) {
        starts[a.B] = T;
        before[a.B] = total;
        if (reports && a.err && (bad_row || !fits || !enough))
            atomicOr(a.err, (bad_row || !fits ? PKV_DEVERR_LENGTH : 0) | (enough ? 0 : PKV_DEVERR_PAGES));
    }
    __syncthreads();
    // (every thread has read lengths, counts and `used`: the ticket, whose answer is needed at the end)
    const int ctas = gridDim.x * gridDim.y;
    int drawn = 0;
    if (ctas > 1 && threadIdx.x == 0)
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(drawn) : "l"(a.ticket) : "memory");
    bool bad_page = false;
    // ---- the new table entries, spread over the grid
    const int64_t entries = (int64_t)total * a.layers, threads = (int64_t)gridDim.x * gridDim.y * kTablesThreads;
    for (int64_t e = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kTablesThreads + threadIdx.x; e < entries; e += threads) {
        const int l = (int)(e / total), k = (int)(e - (int64_t)l * total);
        const int b = find_row(before, a.B, k);
        int id = a.pages[used + e];
        if (id < 0 || id >= a.num_pages) {
            id = -1;
            bad_page = true;
        }
        a.bt[((size_t)l * a.B + b) * a.max_blocks + pages_of(lens[b]) + (k - before[b])] = id;
    }
    // ---- positions and slots: a thread takes one token of the tile in several layers
    const int t = blockIdx.x * a.tile + (threadIdx.x & (a.tile - 1));
    const int step = kTablesThreads / a.tile * a.layer_ctas;
    if (t < a.max_tokens) {
        int b = 0, p = 0, page = 0;
        bool mine = false;     // the token's page is a new one
        int64_t list = 0;      // its place in layer 0
        const bool live = t < T;
        if (live) {
            b = find_row(starts, a.B, t);
            p = lens[b] + (t - starts[b]);
            page = p / kPage;
            const int had = pages_of(lens[b]);
            mine = page >= had;
            list = (int64_t)used + before[b] + (page - had);
        }
        const int l0 = blockIdx.y * (kTablesThreads / a.tile) + threadIdx.x / a.tile;
        if (l0 == 0)
            a.pos[t] = p;
        // where the layers' page ids are, one `next` behind the other
        const int32_t *src = mine ? a.pages + list : a.bt + (size_t)b * a.max_blocks + page;
        const int64_t next = mine ? total : (int64_t)a.B * a.max_blocks;
        for (int l = l0; l < a.layers; l += kLayersAtOnce * step) {
            int id[kLayersAtOnce];
#pragma unroll
            for (int i = 0; i < kLayersAtOnce; ++i)
                id[i] = live && l + i * step < a.layers ? src[(l + i * step) * next] : -1;
#pragma unroll
            for (int i = 0; i < kLayersAtOnce; ++i) {
                const bool ok = id[i] >= 0 && id[i] < a.num_pages;
                if (l + i * step < a.layers) {
                    bad_page |= live && !ok;
                    a.slots[(size_t)(l + i * step) * a.max_tokens + t] = ok ? (int64_t)id[i] * kPage + p % kPage : -1;
                }
            }
        }
    }
    if (bad_page && a.err)
        atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
    // ---- what may be the call's inputs, once every CTA has read them
    if (ctas > 1) {
        __shared__ int last;
        if (threadIdx.x == 0) {
            last = drawn == ctas - 1;
            if (last)
                *a.ticket = 0;
        }
        __syncthreads();
        if (!last)
            return;
    }
    for (int b = threadIdx.x; b <= a.B; b += kTablesThreads) {
        a.starts[b] = starts[b];
        if (b < a.B)
            a.lens_out[b] = lens[b] + (starts[b + 1] - starts[b]);
    }
    if (threadIdx.x == 0)
        *a.used_out = used + total * a.layers;
}

bool tables_args_ok(int B) { return B >= 1 && B <= kMaxRows; }

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_chunk_tables_workspace_bytes(int B) { return pkv::tables_args_ok(B) ? 16 : 0; }

extern "C" int pkv_chunk_tables(const pkv_pool *pool, const int32_t *seq_lens_dev, const int32_t *new_dev, int B,
                                int32_t *bt_dev, int max_blocks, int layers, const int32_t *pages_dev, int pages,
                                const int32_t *pages_used_dev, int32_t *pages_used_out, int max_tokens,
                                int32_t *starts_out, int32_t *seq_lens_out, int32_t *pos_out, int64_t *slots_out,
                                void *workspace, size_t workspace_bytes, int32_t *dev_err_flag, void *cuda_stream)
{
    using namespace pkv;
    if (!pool || !seq_lens_dev || !new_dev || !bt_dev || !pages_used_dev || !pages_used_out || !starts_out ||
        !seq_lens_out || !pos_out || !slots_out || !workspace || (pages > 0 && !pages_dev))
        return PKV_ERR_INVALID_ARG;
    if (!tables_args_ok(B) || max_blocks < 1 || max_blocks > (1 << 20) || layers < 1 || layers > 65535 || pages < 0 ||
        max_tokens < 1 || max_tokens > INT32_MAX / 2)
        return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(workspace) & 15u) || (reinterpret_cast<uintptr_t>(slots_out) & 7u))
        return PKV_ERR_INVALID_ARG;
    if (workspace_bytes < pkv_chunk_tables_workspace_bytes(B))
        return PKV_ERR_WORKSPACE_TOO_SMALL;
    TablesArgs a;
    a.lens = seq_lens_dev;
    a.fresh = new_dev;
    a.B = B;
    a.bt = bt_dev;
    a.max_blocks = max_blocks;
    a.layers = layers;
    a.pages = pages_dev;
    a.num_listed = pages;
    a.used = pages_used_dev;
    a.used_out = pages_used_out;
    a.max_tokens = max_tokens;
    a.starts = starts_out;
    a.lens_out = seq_lens_out;
    a.pos = pos_out;
    a.slots = slots_out;
    a.num_pages = pool->num_pages;
    a.ticket = static_cast<int *>(workspace);
    a.err = dev_err_flag;
    // one token a thread while that fills the GPU; fewer tokens leave threads and CTAs for the layers
    a.tile = 1;
    while (a.tile < kTablesThreads && a.tile < max_tokens)
        a.tile *= 2;
    const int tiles = (max_tokens + a.tile - 1) / a.tile, per_cta = kTablesThreads / a.tile;
    a.layer_ctas = std::max(1, std::min(kTablesCtas / tiles, (layers + per_cta - 1) / per_cta));
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    pages_written(pool, s);  // a decode launch behind it may read these lengths and tables
    return launch_kernel(chunk_tables_kernel, dim3(tiles, a.layer_ctas), dim3(kTablesThreads), 0, s, true, a);
}
