// pkv_chunk_run.cuh -- what the kernels of the attention of chunks share: their arguments, the pieces of work, the
// plan that every CTA makes for itself and the warp that hands its pieces to the others.  Not part of the ABI.
//
// A kernel is described by Run: kThreads, kConsumers (warps that go through the pieces), kSingles (it takes the
// sequences' single tokens, and those alone) and costs().
#pragma once

#include "pkv_chunk_plan.cuh"
#include "pkv_tc.cuh"

namespace pkv {
namespace chunk {

using namespace dev;
using plan::Costs;
using plan::PageList;

constexpr int kMaxRows = 4096;       // sequences of a call
constexpr int kSms = 152;
// Pieces that are handed out ahead.  (The loader is four key tiles in front, of four pieces where they are short: with 4, 16
// prompts of 2048 take 213 us where this takes 196, with 8 200.)
constexpr int kItems = 16;
constexpr int kTokenRow = kHq * kD;  // elements of a token's query rows
constexpr int kPagesOfTile = plan::kTileTokens / kPage;

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
    int *tickets;    // [CTA][2] of cut items that begin there, zero between launches
    int *arrived;    // what came before this call's first kernel has ended; zero between calls (see launch_singles)
    float2 *part_ml; // partials of cut items: (m, l), and O, of [CTA][went on, begun][rows]
    float *part_o;
    int expire;      // testing aid (PKV_STEP_TEST_EXPIRE_WAIT)
    bool apart;      // single tokens are another kernel's
    bool refuses;    // this kernel writes the zeros of refused rows and reports them
};

// A piece of work, as the scheduler hands it to the other warps.
struct Item {
    int kind;
    int b, g;              // sequence, (first) KV head
    int t0, n, p0;         // first token, tokens, position of the first
    int sink, from, count; // its pages
    int j0, j1, nt;        // key tiles of the piece; of the whole item
    int first, parts, me;  // CTAs that share the item, and this one's place among them
    int plain, plain0, plain1;  // key tiles in which every row attends to every place: below plain, and plain0 .. plain1 - 1
    int pad;
    int64_t row;           // first query row, in elements
    __device__ __forceinline__ int page(int i) const { return i < sink ? i : i - sink + from; }
    __device__ __forceinline__ int loads() const { return (j1 - j0) * (kind == plan::kHeads ? 2 : 1); }
    // A row tile's first token within the item, its tokens, its KV head, and the place among the piece's loads of
    // the piece's j-th key tile.
    __device__ __forceinline__ int token(int s) const { return kind == plan::kPair ? 32 * s : 0; }
    __device__ __forceinline__ int tokens(int s) const { return min(plan::kRowTokens, n - token(s)); }
    __device__ __forceinline__ int order(int s, int j) const { return kind == plan::kHeads ? 2 * j + s : j; }
    __device__ __forceinline__ bool masked(int j) const { return j >= plain && (j < plain0 || j >= plain1); }
    // Loads of the piece before its j-th key tile's first whose tiles are masked.
    __device__ __forceinline__ int masked_loads(int j) const
    {
        const int n = masked_tiles(j0 + j) - masked_tiles(j0);
        return kind == plan::kHeads ? 2 * n : n;
    }
    __device__ __forceinline__ int masked_tiles(int j) const
    {
        return j - min(j, plain) - (min(max(j, plain0), plain1) - plain0);
    }
    __device__ __forceinline__ void find_plain(int window, int sinks)
    {
        const int whole = (p0 + 1) / kPage;  // pages that end at or before the first token
        plain1 = min(count, max(whole + sink - from, 0)) / kPagesOfTile;
        plain = plain0 = 0;
        if (window) {
            plain = min(sink, sinks / kPage) / kPagesOfTile;  // entries from the first page on that the last token's window holds as a whole
            const int entry = max(sink, sink - from + (max(p0 + n - window, 0) + kPage - 1) / kPage);
            plain0 = (entry + kPagesOfTile - 1) / kPagesOfTile;
        }
        plain1 = max(plain1, plain0);
    }
};

// What hands the pieces out, in shared memory; a kernel adds `sums`, the costs of the sequences before each thread's.
struct RunShared {
    uint64_t item_full[kItems], item_empty[kItems];
    int stop;            // a wait gave up
    int taken[2][2];     // [went on, begun][row tile]: the cut item's ticket is drawn
    int64_t length;      // of the line
    int64_t warp_sums[32];
    alignas(16) Item items[kItems];
};

// A bounded wait of a whole warp (see tc::wait_warp).
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *stop)
{
    return tc::wait_warp(bar, parity, stop);
}

// ------------------------------------------------------------------ the plan

struct Row {
    int s0, n, L;
    bool ok;
};

// Sequence b; not ok if its tokens are out of range.
__device__ __forceinline__ Row row_of(const ChunkArgs &a, int b)
{
    Row x;
    x.s0 = a.starts[b];
    const int s1 = a.starts[b + 1];
    x.ok = x.s0 >= 0 && s1 >= x.s0 && s1 <= a.T;
    x.n = x.ok ? s1 - x.s0 : 0;
    x.L = a.lens[b];
    return x;
}

__device__ __forceinline__ bool length_fits(const ChunkArgs &a, const Row &x)
{
    return x.L >= x.n && x.L <= a.max_blocks * kPage;
}

template <class Run>
__device__ __forceinline__ int64_t row_cost(const ChunkArgs &a, const Row &x, const Costs &k)
{
    if (!x.n || !length_fits(a, x))
        return 0;
    if (Run::kSingles ? x.n != 1 : a.apart && x.n == 1)
        return 0;
    if (plan::short_row(x.n, x.L))
        return plan::row_cost<int>(x.n, x.L, a.window, a.sinks, k, Run::kSingles);
    return plan::row_cost<int64_t>(x.n, x.L, a.window, a.sinks, k, Run::kSingles);
}

// All rows zeros.  (Out of line: within the plan, 16 prompts of 2048 took 203.6 us where this takes 200.8.)
static __device__ __noinline__ void refuse_all(uint16_t *out, int T)
{
    const int64_t words = (int64_t)T * (kTokenRow / 8), threads = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < words; i += threads)
        reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
}

// All threads: the prefix sums of the sequences' costs, the rows that are refused.  Starts that are no prefix sums (from
// 0 on, none below the one before, T at most) say nothing about whose a token is, and two sequences may name the same:
// then nothing is worked on and every row is zeros.
template <class Run, class Shared>
__device__ __forceinline__ void make_plan(const ChunkArgs &a, Shared &sh)
{
    const Costs k = Run::costs();
    const int per = (a.B + Run::kThreads - 1) / Run::kThreads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t sum = 0;
    bool bad = false, no_starts = threadIdx.x == 0 && a.starts[0] != 0;
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b >= a.B)
            break;
        const Row x = row_of(a, b);
        no_starts |= !x.ok;
        if (x.n && !length_fits(a, x)) {  // zeros; the CTAs share the tokens
            bad = true;
            for (int t = blockIdx.x; a.refuses && t < x.n; t += gridDim.x)
                for (int i2 = 0; i2 < kHq * kD / 8; ++i2)
                    reinterpret_cast<uint4 *>(a.out + (size_t)(x.s0 + t) * kHq * kD)[i2] = make_uint4(0, 0, 0, 0);
        }
        sum += row_cost<Run>(a, x, k);
    }
    int64_t upto = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, upto, off);
        if (lane >= off)
            upto += y;
    }
    no_starts = __any_sync(kFull, no_starts);
    if (lane == 31)
        sh.warp_sums[warp] = no_starts ? -1 : upto;
    bad = __syncthreads_or(bad || no_starts);
    int64_t before = upto - sum, all = 0;
    no_starts = false;
    for (int w = 0; w < Run::kThreads / 32; ++w) {
        const int64_t of = sh.warp_sums[w];
        if (w < warp)
            before += of;
        all += of;
        no_starts |= of < 0;
    }
    if (no_starts) {  // (all threads of all CTAs alike)
        all = 0;
        if (a.refuses)
            refuse_all(a.out, a.T);
    }
    sh.sums[threadIdx.x] = before;
    if (threadIdx.x == 0) {
        sh.length = all;
        if (bad && a.refuses && blockIdx.x == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_LENGTH);
    }
}

// A piece for the other warps, `n` so far; false if a wait gave up.
__device__ __forceinline__ bool give(RunShared &sh, const Item &it, int &n)
{
    const int at = n % kItems;
    if (n >= kItems && !wait_for(&sh.item_empty[at], (n / kItems - 1) & 1, &sh.stop))
        return false;
    if ((threadIdx.x & 31) == 0) {
        sh.items[at] = it;
        tc::mbar_arrive(&sh.item_full[at]);
    }
    __syncwarp();
    ++n;
    return true;
}

// The pieces of this CTA's run, in order, by a whole warp, given to the others; or (`over`: something gave up) the
// tickets of cut items that were not drawn, so that the next call finds zeros.
template <class Run, class I, class Shared>
__device__ __forceinline__ void pieces_of(const ChunkArgs &a, Shared &sh, bool over)
{
    int given = 0;
    const Costs k = Run::costs();
    const plan::Line<I> line((I)sh.length, gridDim.x, Run::kLeast);
    const int lane = threadIdx.x & 31, per = (a.B + Run::kThreads - 1) / Run::kThreads;
    const bool work = line.length > 0 && (int)blockIdx.x < line.ctas;
    const I x0 = work ? line.border(blockIdx.x) : 0, x1 = work ? line.border(blockIdx.x + 1) : 0;
    I x = x0;
    while (x < x1) {
        // the thread whose sequences hold x (the last whose sum is not above it), and the sequence
        int lo = 0, hi = Run::kThreads;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sh.sums[mid] <= x)
                lo = mid;
            else
                hi = mid;
        }
        const int b0 = lo * per + lane;
        const I mine = lane < per && b0 < a.B ? (I)row_cost<Run>(a, row_of(a, b0), k) : 0;
        I upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const I y = __shfl_up_sync(kFull, upto, off);
            if (lane >= off)
                upto += y;
        }
        const I sum = (I)sh.sums[lo];
        const unsigned behind = __ballot_sync(kFull, sum + upto > x);
        if (!behind)
            break;  // (not reached: the sums add up to the length)
        const int at = __ffs(behind) - 1, b = lo * per + at;
        const I begin = sum + __shfl_sync(kFull, upto - mine, at), end = sum + __shfl_sync(kFull, upto, at);
        const Row row = row_of(a, b);
        const plan::Sequence<I> seq(row.n, row.L - row.n, a.window, a.sinks, k);
        const I head = Run::kSingles ? 0 : seq.head_cost(), rest = Run::kSingles ? 0 : seq.rest_cost(k);
        const I single = Run::kSingles ? seq.single_cost(k) : 0;
        // the item that holds x: its kind, (first) KV head, pair, and where it begins
        I s, y = x - begin;
        int kind = plan::kSingle, g, r = 0;
        if (Run::kSingles) {
            g = plan::eighth(y, single);
            s = begin + g * single;
        } else if (y < kHkv * head) {
            kind = plan::kPair;
            g = plan::eighth(y, head);
            y -= g * head;
            r = seq.pairs - 1;
            if (y < seq.before(r)) {  // the last r that does not begin behind y, by 32 tries at a time
                int from = 0, to = r;
                while (to - from > 1) {
                    const int step = (to - from + 31) / 32, probe = from + (lane + 1) * step;
                    const int n = __popc(__ballot_sync(kFull, probe < to && seq.before(probe) <= y));
                    from += n * step;
                    to = min(to, from + step);
                }
                r = from;
            }
            s = begin + g * head + seq.before(r);
        } else {
            kind = plan::kHeads;
            const int h = plan::eighth((I)(y - kHkv * head), rest);
            g = 2 * h;
            s = begin + kHkv * head + h * rest;
        }
        while (x < x1 && x < end) {
            Item it;
            it.kind = kind;
            it.b = b;
            it.g = g;
            int token = 0;
            PageList pages;
            if (kind == plan::kPair) {
                token = 64 * r;
                it.n = min(64, row.n - token);
                pages = seq.pair_pages(r);
            } else if (kind == plan::kHeads) {
                token = 64 * seq.pairs;
                it.n = row.n - token;
                pages = seq.rest_pages();
            } else {
                it.n = 1;
                pages = seq.single_pages();
            }
            it.t0 = row.s0 + token;
            it.p0 = row.L - row.n + token;
            it.sink = pages.sink;
            it.from = pages.from;
            it.count = pages.count;
            it.nt = pages.tiles();
            const int tile = k.tile[it.kind], item = k.item[it.kind];
            const I next = s + (I)it.nt * tile + item;
            if (x0 <= s && next <= x1) {  // (most: the whole item)
                it.j0 = it.me = 0;
                it.j1 = it.nt;
                it.first = blockIdx.x;
                it.parts = 1;
            } else {
                it.j0 = x0 <= s ? 0 : plan::cut(x0 - s, it.nt, tile, item);
                it.j1 = plan::cut(x1 - s, it.nt, tile, item);
                const plan::Parts parts = plan::parts_of(line, s, it.nt, tile, item);
                it.first = parts.first;
                it.parts = parts.count;
                it.me = blockIdx.x - parts.first;
            }
            it.find_plain(a.window, a.sinks);
            it.row = ((int64_t)it.t0 * kHq + it.g * kGroup) * kD;
            if (it.j0 < it.j1) {
                if (!over) {
                    if (!give(sh, it, given))
                        return;
                } else if (it.parts > 1 && lane == 0) {
                    for (int r = 0; r < (Run::kSingles ? 1 : 2); ++r)
                        if (!sh.taken[it.me == 0][r] && atomicAdd(&a.tickets[it.first * 2 + r], 1) == it.parts - 1)
                            a.tickets[it.first * 2 + r] = 0;
                }
            }
            x = s = next;
            if (kind == plan::kPair && ++r < seq.pairs)
                continue;
            r = 0;
            g += kind == plan::kHeads ? 2 : 1;
            if (kind == plan::kPair && g == kHkv) {
                kind = plan::kHeads;
                g = 0;
            }
        }
    }
    if (!over) {
        Item end = {};
        (void)give(sh, end, given);
    }
}

template <class Run, class Shared>
__device__ __noinline__ void pieces(const ChunkArgs &a, Shared &sh, bool over)
{
    if (sh.length < 1 << 30)
        pieces_of<Run, int>(a, sh, over);
    else
        pieces_of<Run, int64_t>(a, sh, over);
}

// The items in order, as a warp of another role goes through them; one is held until it is let go.
struct Feed {
    RunShared &sh;
    int n = 0;
    __device__ __forceinline__ explicit Feed(RunShared &s) : sh(s) {}
    // The item `ahead` of the current one, or null at the end (or after a wait that gave up).
    __device__ __forceinline__ const Item *look(int ahead = 0)
    {
        const int at = (n + ahead) % kItems;
        if (!wait_for(&sh.item_full[at], ((n + ahead) / kItems) & 1, &sh.stop))
            return nullptr;
        return sh.items[at].kind == plan::kEnd ? nullptr : &sh.items[at];
    }
    __device__ __forceinline__ void let_go()
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            tc::mbar_arrive(&sh.item_empty[n % kItems]);
        ++n;
    }
};


inline bool chunk_args_ok(int B, int T) { return B >= 1 && B <= kMaxRows && T >= 1 && T <= INT32_MAX / 16; }

// A row's (m, l) of a part with a bad page id: what no scores make (l is a sum of weights; m becomes +inf by itself
// where a score is).
__device__ __forceinline__ float2 bad_part() { return make_float2(-INFINITY, -1.f); }
__device__ __forceinline__ bool is_bad_part(float l) { return l < 0.f; }

// Sums and rounded quotients: nothing attended to is zeros, something not finite stays so.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }

// ------------------------------------------------------------------ single tokens (pkv_chunk_single.cu)

constexpr int kSingleCtas = kSms * 4;

struct SingleWorkspace {
    size_t tickets, ml, o;
    size_t total() const { return tickets + ml + o; }
};

inline SingleWorkspace single_workspace()
{
    SingleWorkspace w;
    w.tickets = align256((size_t)kSingleCtas * 2 * sizeof(int));
    w.ml = align256((size_t)kSingleCtas * 2 * kGroup * sizeof(float2));
    w.o = (size_t)kSingleCtas * 2 * kGroup * kD * sizeof(float);
    return w;
}

// The sequences that bring one token, by a kernel of their own; `follows`: behind the kernel of the others, beside which
// it runs (refused rows are dealt with there).  It begins when the other's CTAs have waited for what came before,
// lengths, queries and pages among it.  Of a launch that another one waited for, the programming model promises nothing to
// a grid that does not wait itself; so the other's first CTA hands its wait on: a release store to `arrived` before it
// lets this kernel begin, which every CTA here acquires.  A CTA that finds nothing there waits for the other kernel
// itself.  This kernel's first CTA does that at its end in any case, because what comes behind waits for this kernel
// alone, and takes the mark back then: CTAs that begin later have nothing left to wait for.
int launch_singles(const pkv_pool *pool, ChunkArgs a, void *workspace, cudaStream_t s, bool pdl, bool follows);

}  // namespace chunk
}  // namespace pkv
