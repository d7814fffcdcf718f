// pkv_chunk.cu -- causal attention of a step's new tokens over their sequences' pages.
//
//     out[t][h] = sum_j softmax_j(scale * q[t][h] . K_j) V_j,   j <= p(t), and j > p(t) - window or j < sinks.
//
// 32 tokens and the 4 query heads of a KV head are 128 rows that meet the same keys: S = Q K^T and O += P V
// on the tensor cores (tcgen05), Q, S, P and O in tensor memory, K and V in shared memory as TMA brought the
// pages.  A CTA has two such row tiles at a time, each with four softmax warps (a thread a row) and an issuer
// warp, so that one's products fill the other's exponentials.  A sequence's single new token is 4 rows: its
// pages go through warp-level products (the decode kernels' policies), a page a warp, from the same ring of
// stages.  pkv_chunk_plan.cuh says how the work is cut into one run for every CTA.
//
// Masks: only tiles in which some row does not attend to some token (the last ones, and a window's
// first) are masked, by 64 bits a row and half tile.  A weight of 0 times a value that is not finite would
// not be 0, so in those tiles values that nobody attends to are cleared in shared memory, and those that are not
// finite too: rows that attend to one get NaN in its dimension at the end.
#include <cmath>

#include "pkv_chunk_plan.cuh"
#include "pkv_tiles.cuh"

namespace pkv {
namespace {

using namespace dev;
using namespace tiles;
using plan::Costs;
using plan::PageList;

constexpr int kMaxRows = 4096;       // sequences of a call
constexpr int kSms = 152;
constexpr int kStages = 4, kRaws = 2, kItems = 4;
constexpr int kLoader = 8, kIssuer = 9, kScheduler = 11, kConverter = 12;   // warps: 2 x 4 softmax, ...
constexpr int kConverters = 4;
constexpr int kTeam = 8;             // warps of a single token's pages
constexpr int kOnesSize = 16 * 128;  // BF16 pages: 16 rows of ones, for the sums
constexpr int kCols = 512;           // tensor memory, all of it
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384, kColL = 448;  // + 128 / 64 / 32 / 16 for the second row tile

constexpr int chunk_threads(bool fp8) { return fp8 ? (kConverter + kConverters) * 32 : kConverter * 32; }
constexpr int consumers(bool fp8) { return fp8 ? 8 + 3 + kConverters : 8 + 3; }

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
    int *tickets;    // [CTA][row tile], zero between launches
    float2 *part_ml; // [CTA][went on, begun][row tile][128] (m, l)
    float *part_o;   // [CTA][went on, begun][row tile][128][64]
    int expire;      // testing aid (PKV_STEP_TEST_EXPIRE_WAIT)
};

// A piece of work, as the scheduler hands it to the other warps.
struct Item {
    int kind;
    int b, g;              // sequence, (first) KV head
    int t0, n, p0;         // first token, tokens, position of the first
    int sink, from, count; // its pages
    int j0, j1, nt;        // key tiles of the piece; of the whole item
    int first, parts, me;  // CTAs that share the item, and this one's place among them
    int pad;
    __device__ __forceinline__ int page(int i) const { return i < sink ? i : i - sink + from; }
    __device__ __forceinline__ int loads() const { return (j1 - j0) * (kind == plan::kHeads ? 2 : 1); }
    // A row tile's first token within the item, its tokens, its KV head, and the place among the piece's loads of
    // the piece's j-th key tile.
    __device__ __forceinline__ int token(int s) const { return kind == plan::kPair ? 32 * s : 0; }
    __device__ __forceinline__ int tokens(int s) const { return min(plan::kRowTokens, n - token(s)); }
    __device__ __forceinline__ int head(int s) const { return kind == plan::kHeads ? g + s : g; }
    __device__ __forceinline__ int order(int s, int j) const { return kind == plan::kHeads ? 2 * j + s : j; }
    // Some row of the item does not attend to some place of key tile j.
    __device__ __forceinline__ bool masked(int j, int window) const
    {
        const int i = j * kTilePages;
        return i + kTilePages > count || page(i + kTilePages - 1) * kPage + kPage - 1 > p0 ||
               (window && (i < sink || page(i) * kPage < p0 + n - window));
    }
};

// A value row that holds something not finite: the load it belongs to, and which dimensions.
struct Poison {
    int load;
    uint32_t lo, hi;
};

struct ChunkShared {
    uint64_t full[kStages], empty[kStages];      // a stage holds its pages / has been read by all
    uint64_t raw_full[kRaws], raw_empty[kRaws];  // the same of the raw units
    uint64_t s_full[2][2], p_full[2][2];         // [row tile][half]: scores are in tensor memory / weights are
    uint64_t o_step[2];                          // one more product of weights and values is done
    uint64_t q_full[2], o_full[2];               // once an item: the queries are in / its last product is done
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t group[3];                           // row tile s's warps (2: all eight) have come so far
    uint64_t drained[2];
    uint32_t tmem;
    int stop;                                    // a wait gave up
    int bad[kStages], raw_bad[kRaws];            // the tile has a bad page id
    int noted[2];                                // the last load of row tile s with notes on values (see Poison)
    int last[3];                                 // group: this CTA finished the item last
    int taken[2][2];                             // [went on, begun][row tile]: the cut item's ticket is drawn
    int64_t length;                              // of the line
    int64_t warp_sums[16];
    alignas(16) Item items[kItems];
    Poison poison[kStages][kTilePages * kPage];
    alignas(16) float states[kTeam][kStateFloats];
    int64_t sums[512];                           // costs of the sequences before each thread's
    float scales[kStages][kScales];              // (FP8)
};

// ------------------------------------------------------------------ the plan

template <bool FP8>
__device__ __forceinline__ Costs costs()
{
    // in eighths of the time of a BF16 key tile of two row tiles
    return FP8 ? Costs{{0, 14, 16, 3}, {0, 30, 30, 8}} : Costs{{0, 8, 9, 5}, {0, 24, 24, 8}};
}
constexpr int kLeastCost = 64;  // of a CTA's run

struct Row {
    int s0, n, L;
    bool ok;
};

// Sequence b; not ok if its tokens or its length are out of range.
__device__ __forceinline__ Row row_of(const ChunkArgs &a, int b)
{
    Row x;
    x.s0 = a.starts[b];
    const int s1 = a.starts[b + 1];
    x.ok = x.s0 >= 0 && s1 >= x.s0 && s1 <= a.T;
    x.n = x.ok ? s1 - x.s0 : 0;
    x.L = x.n ? a.lens[b] : 0;
    return x;
}

__device__ __forceinline__ bool length_fits(const ChunkArgs &a, const Row &x)
{
    return x.L >= x.n && x.L <= a.max_blocks * kPage;
}

__device__ __forceinline__ int64_t row_cost(const ChunkArgs &a, const Row &x, const Costs &k)
{
    return x.n && length_fits(a, x) ? plan::Sequence(x.n, x.L - x.n, a.window, a.sinks, k).cost(k) : 0;
}

// All threads: the prefix sums of the sequences' costs, the rows that are refused.
template <bool FP8>
__device__ __forceinline__ void make_plan(const ChunkArgs &a, ChunkShared &sh)
{
    constexpr int kThreadsHere = chunk_threads(FP8);
    const Costs k = costs<FP8>();
    const int per = (a.B + kThreadsHere - 1) / kThreadsHere;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t sum = 0;
    bool bad = threadIdx.x == 0 && a.starts[0] != 0;
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b >= a.B)
            break;
        const Row x = row_of(a, b);
        bad |= !x.ok;
        if (x.n && !length_fits(a, x)) {  // zeros; the CTAs share the tokens
            bad = true;
            for (int t = blockIdx.x; t < x.n; t += gridDim.x)
                for (int i2 = 0; i2 < kHq * kD / 8; ++i2)
                    reinterpret_cast<uint4 *>(a.out + (size_t)(x.s0 + t) * kHq * kD)[i2] = make_uint4(0, 0, 0, 0);
        }
        sum += row_cost(a, x, k);
    }
    int64_t upto = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, upto, off);
        if (lane >= off)
            upto += y;
    }
    if (lane == 31)
        sh.warp_sums[warp] = upto;
    bad = __syncthreads_or(bad);
    int64_t before = upto - sum, all = 0;
    for (int w = 0; w < kThreadsHere / 32; ++w) {
        if (w < warp)
            before += sh.warp_sums[w];
        all += sh.warp_sums[w];
    }
    sh.sums[threadIdx.x] = before;
    if (threadIdx.x == 0) {
        sh.length = all;
        if (bad && blockIdx.x == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_LENGTH);
    }
}

// The pieces of this CTA's run, in order, by a whole warp; `take(item)` may end it by returning false.
template <bool FP8, class Take>
__device__ __forceinline__ void for_each_piece(const ChunkArgs &a, const ChunkShared &sh, const Take &take)
{
    constexpr int kThreadsHere = chunk_threads(FP8);
    const Costs k = costs<FP8>();
    const plan::Line line = plan::line_of(sh.length, gridDim.x, kLeastCost);
    if (line.length == 0 || (int)blockIdx.x >= line.ctas)
        return;
    const int lane = threadIdx.x & 31, per = (a.B + kThreadsHere - 1) / kThreadsHere;
    const int64_t x0 = line.border(blockIdx.x), x1 = line.border(blockIdx.x + 1);
    int64_t x = x0;
    while (x < x1) {
        // the thread whose sequences hold x (the last whose sum is not above it), and the sequence
        int lo = 0, hi = kThreadsHere;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sh.sums[mid] <= x)
                lo = mid;
            else
                hi = mid;
        }
        const int b0 = lo * per + lane;
        const int64_t mine = lane < per && b0 < a.B ? row_cost(a, row_of(a, b0), k) : 0;
        int64_t upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(kFull, upto, off);
            if (lane >= off)
                upto += y;
        }
        const unsigned behind = __ballot_sync(kFull, sh.sums[lo] + upto > x);
        if (!behind)
            return;  // (not reached: the sums add up to the length)
        const int at = __ffs(behind) - 1, b = lo * per + at;
        const int64_t begin = sh.sums[lo] + __shfl_sync(kFull, upto - mine, at), end = sh.sums[lo] + __shfl_sync(kFull, upto, at);
        const Row row = row_of(a, b);
        const plan::Sequence seq(row.n, row.L - row.n, a.window, a.sinks, k);
        const int64_t head = seq.head_cost(), rest = seq.rest_cost(k), single = seq.single_cost(k);
        while (x < x1 && x < end) {
            Item it;
            PageList pages;
            int64_t s;  // where the item begins
            int64_t y = x - begin;
            int token = 0;
            it.b = b;
            if (row.n == 1) {
                it.kind = plan::kSingle;
                it.g = (int)(y / single);
                s = begin + it.g * single;
                it.n = 1;
                pages = seq.single_pages();
            } else if (y < kHkv * head) {
                it.kind = plan::kPair;
                it.g = (int)(y / head);
                y -= it.g * head;
                int r = seq.pairs - 1;
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
                s = begin + it.g * head + seq.before(r);
                token = 64 * r;
                it.n = min(64, row.n - token);
                pages = seq.pair_pages(r);
            } else {
                it.kind = plan::kHeads;
                const int h = (int)((y - kHkv * head) / rest);
                it.g = 2 * h;
                s = begin + kHkv * head + h * rest;
                token = 64 * seq.pairs;
                it.n = row.n - token;
                pages = seq.rest_pages();
            }
            it.t0 = row.s0 + token;
            it.p0 = row.L - row.n + token;
            it.sink = pages.sink;
            it.from = pages.from;
            it.count = pages.count;
            it.nt = pages.tiles();
            const int tile = k.tile[it.kind], over = k.item[it.kind];
            it.j0 = x0 <= s ? 0 : plan::cut(x0 - s, it.nt, tile, over);
            it.j1 = plan::cut(x1 - s, it.nt, tile, over);
            const plan::Parts parts = plan::parts_of(line, s, it.nt, tile, over);
            it.first = parts.first;
            it.parts = parts.count;
            it.me = blockIdx.x - parts.first;
            it.pad = 0;
            if (it.j0 < it.j1 && !take(it))
                return;
            x = s + (int64_t)it.nt * tile + over;
        }
    }
}

template <bool FP8>
__device__ __forceinline__ void scheduler(const ChunkArgs &a, ChunkShared &sh)
{
    int n = 0;
    const auto give = [&](const Item &it) {
        const int at = n % kItems;
        if (n >= kItems && !tc::wait_warp(&sh.item_empty[at], (n / kItems - 1) & 1, &sh.stop))
            return false;
        if ((threadIdx.x & 31) == 0) {
            sh.items[at] = it;
            tc::mbar_arrive(&sh.item_full[at]);
        }
        __syncwarp();
        ++n;
        return true;
    };
    bool open = true;
    for_each_piece<FP8>(a, sh, [&](const Item &it) { return open = give(it); });
    if (open) {
        Item end = {};
        (void)give(end);
    }
}

// The items in order, as a warp of another role goes through them; one is held until it is let go.
struct Feed {
    ChunkShared &sh;
    int n = 0;
    __device__ __forceinline__ explicit Feed(ChunkShared &s) : sh(s) {}
    // The item `ahead` of the current one, or null at the end (or after a wait that gave up).
    __device__ __forceinline__ const Item *look(int ahead = 0)
    {
        const int at = (n + ahead) % kItems;
        if (!tc::wait_warp(&sh.item_full[at], ((n + ahead) / kItems) & 1, &sh.stop))
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

__device__ __forceinline__ void arrive_n(uint64_t *bar, int n)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}

// A stage is free after kTeam arrivals: those of the team's warps, or the row tiles' last products and what whoever
// fills the stage gives in advance for the others.
__device__ __forceinline__ int given_in_advance(int kind)
{
    return kind == plan::kPair ? kTeam - 2 : kTeam - 1;
}

// ------------------------------------------------------------------ loader

// The pages of every piece's key tiles into the ring of stages (FP8 row tiles: of raw units).  A tile that
// the pages do not fill repeats the last one (its places are masked); a bad page id is replaced by page 0
// and the tile marked.
template <bool FP8>
__device__ __forceinline__ void loader(const CUtensorMap *tmap, const ChunkArgs &a, uint8_t *stages, uint8_t *raws,
                                       ChunkShared &sh)
{
    const int lane = threadIdx.x & 31;
    uint64_t shared_policy;  // row tiles' pages are read by several CTAs: no eviction hint
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(shared_policy));
    const uint64_t once_policy = l2_evict_first_policy();
    Feed feed(sh);
    int seq = 0, raw = 0;  // stages and raw units filled so far
    bool go = true;
    for (const Item *p; go && (p = feed.look()) != nullptr; feed.let_go()) {
        const Item x = *p;
        const int32_t *row = a.bt + (size_t)x.b * a.max_blocks;
        const bool single = x.kind == plan::kSingle, through_raw = FP8 && !single;
        const int heads = x.kind == plan::kHeads ? 2 : 1;
        const uint64_t policy = single ? once_policy : shared_policy;
        if (FP8 && single)  // the converters are done with every stage before
            for (int i = max(raw - kRaws, 0); go && i < raw; ++i)
                go = tc::wait_warp(&sh.raw_empty[i % kRaws], (i / kRaws) & 1, &sh.stop);
        int id4 = 0;  // lane l: the id of page l of the current run of 4 key tiles
        unsigned bad4 = 0;
        for (int j = x.j0; j < x.j1 && go; ++j) {
            const int in4 = (j - x.j0) & 3;
            if (in4 == 0) {
                id4 = row[x.page(min(j * kTilePages + lane, x.count - 1))];
                const bool out = id4 < 0 || id4 >= a.num_pages;
                bad4 = __ballot_sync(kFull, out);
                if (out)
                    id4 = 0;
            }
            const int id = __shfl_sync(kFull, id4, in4 * kTilePages + lane % kTilePages);
            const int bad = (bad4 >> (in4 * kTilePages)) & ((1u << kTilePages) - 1);
            for (int h = 0; h < heads && go; ++h) {
                const int st = through_raw ? raw % kRaws : seq % kStages;
                uint64_t *full = through_raw ? &sh.raw_full[st] : &sh.full[st];
                if (through_raw) {
                    if (raw >= kRaws && !tc::wait_warp(&sh.raw_empty[st], (raw / kRaws - 1) & 1, &sh.stop)) {
                        go = false;
                        break;
                    }
                } else if (seq >= kStages && !tc::wait_warp(&sh.empty[st], (seq / kStages - 1) & 1, &sh.stop)) {
                    go = false;
                    break;
                }
                fence_proxy_async_smem();  // (the place's readers and writers so far were threads)
                const int size = FP8 ? kRawSize : kStageSize;
                uint8_t *dst = through_raw ? raws + st * kRawSize : stages + st * kStageSize;
                if (lane == 0) {
                    (through_raw ? sh.raw_bad : sh.bad)[st] = bad;
                    if (!through_raw && !single)
                        arrive_n(&sh.empty[st], given_in_advance(x.kind));
                    if (FP8 && single)
                        arrive_n(full, kConverters - 1);
                    mbar_arrive_expect_tx(full, size);
                }
                __syncwarp();
                if (lane < kTilePages) {
                    if (FP8)
                        fp8::tma_load_unit(dst + lane * kFp8Unit, tmap, full, x.g + h, id, policy);
                    else
                        tma_load_page_head(dst + lane * kStageBytes, tmap, full, x.g + h, id, policy);
                }
                if (through_raw)
                    ++raw;
                ++seq;
            }
        }
    }
    if (*(volatile int *)&sh.stop) {  // let the copies in flight land (bounded)
        for (int i = max(raw - kRaws, 0); i < raw; ++i)
            (void)mbar_wait_warp(&sh.raw_full[i % kRaws], (i / kRaws) & 1);
        for (int i = max(seq - kStages, 0); i < seq; ++i)  // (stages that nobody filled run out of polls)
            (void)mbar_wait_warp(&sh.full[i % kStages], (i / kStages) & 1, FP8 ? 1u << 16 : kWaitLimit);
    }
}

// ------------------------------------------------------------------ converters (FP8 row tiles; 128 threads)

__device__ __forceinline__ void converter(const ChunkArgs &a, const uint8_t *raws, uint8_t *stages, ChunkShared &sh)
{
    const int t = threadIdx.x - kConverter * 32, lane = threadIdx.x & 31;
    Feed feed(sh);
    int seq = 0, raw = 0;
    for (const Item *x; (x = feed.look()) != nullptr; feed.let_go()) {
        const int n = x->loads(), kind = x->kind;
        if (kind == plan::kSingle) {
            seq += n;
            continue;
        }
        for (int i = 0; i < n; ++i, ++seq, ++raw) {
            const int rs = raw % kRaws, st = seq % kStages;
            if (!tc::wait_warp(&sh.raw_full[rs], (raw / kRaws) & 1, &sh.stop) ||
                (seq >= kStages && !tc::wait_warp(&sh.empty[st], (seq / kStages - 1) & 1, &sh.stop)))
                return;
            convert_tile(raws + rs * kRawSize, stages + st * kStageSize, sh.scales[st], a.scale_log2, t);
            if (t == 0) {
                sh.bad[st] = sh.raw_bad[rs];
                arrive_n(&sh.empty[st], given_in_advance(kind));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&sh.raw_empty[rs]);
                tc::mbar_arrive(&sh.full[st]);
            }
        }
    }
}

// ------------------------------------------------------------------ issuers

// Each row tile has an issuer warp of its own, so that one's waits pass while the other's products run.
template <bool FP8>
__device__ __forceinline__ void issuer(uint8_t *stages, const uint8_t *ones, ChunkShared &sh, uint32_t tmem, int s)
{
    const uint32_t base = smem_addr(stages), one = smem_addr(ones), tl = tmem + kColL + s * 16;
    const uint32_t ts = tmem + kColS + s * 128, to = tmem + kColO + s * 64, tq = tmem + kColQ + s * 32;
    Feed feed(sh);
    int loaded = 0, done = 0, used = 0;  // loads of earlier pieces, key tiles of this row tile, pieces with row tiles
    for (const Item *p; (p = feed.look()) != nullptr; feed.let_go()) {
        const Item x = *p;
        if (x.kind != plan::kSingle) {
            const int nt = x.j1 - x.j0;
            const auto scores = [&](int j, int h) {
                const int seq = loaded + x.order(s, j), st = seq % kStages;
                if (h == 0) {
                    if (!tc::wait_warp(&sh.full[st], (seq / kStages) & 1, &sh.stop))
                        return false;
                    tc::fence_after();
                }
                issue_scores(base + st * kStageSize + h * 1024, ts + h * kHalf, tq, &sh.s_full[s][h]);
                return true;
            };
            const auto output = [&](int j, int h) {
                if (!tc::wait_warp(&sh.p_full[s][h], (done + j) & 1, &sh.stop))
                    return false;
                tc::fence_after();
                const int st = (loaded + x.order(s, j)) % kStages;
                const uint32_t v = base + st * kStageSize + kTileBytes + h * 1024, pw = ts + h * kHalf;
                uint64_t *empty = h == 1 ? &sh.empty[st] : nullptr;
                uint64_t *last = h == 1 && j + 1 == nt ? &sh.o_full[s] : nullptr;
                if (j == 0 && h == 0)
                    issue_output<true, !FP8>(v, to, pw, one, tl, empty, 1, &sh.o_step[s], last);
                else
                    issue_output<false, !FP8>(v, to, pw, one, tl, empty, 1, &sh.o_step[s], last);
                return true;
            };
            bool go = tc::wait_warp(&sh.q_full[s], used & 1, &sh.stop);
            tc::fence_after();
            go = go && scores(0, 0) && scores(0, 1);
            for (int j = 0; j < nt && go; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (go) {
                        go = output(j, h);
                        if (go && j + 1 < nt)
                            go = scores(j + 1, h);
                    }
            if (!go)
                break;
            ++used;
            done += nt;
        }
        loaded += x.loads();
    }
    if (*(volatile int *)&sh.stop) {  // let the products in flight end (bounded)
        if (tc::elect())
            tc::commit(&sh.drained[s]);
        __syncwarp();
        (void)mbar_wait_warp(&sh.drained[s], 0);
    }
}

// ------------------------------------------------------------------ softmax

// The low n bits, n of 0..8 after clamping.
__device__ __forceinline__ uint32_t low_bits(int n) { return (1u << min(max(n, 0), 8)) - 1; }

// What a row at position p attends to in half hf of key tile j.
__device__ __forceinline__ ColumnBits columns(const Item &x, int j, int hf, int p, int window, int sinks)
{
    uint32_t w[2] = {0, 0};
    const int lo = window ? max(p + 1 - window, 0) : 0;
#pragma unroll
    for (int i = 0; i < kTilePages; ++i) {
        const int at = j * kTilePages + i, first = x.page(at) * kPage + 8 * hf;
        uint32_t bits = low_bits(p + 1 - first) & (~low_bits(lo - first) | low_bits(sinks - first));
        if (at >= x.count)
            bits = 0;
        w[i / 4] |= bits << (i % 4 * 8);
    }
    return {w[0], w[1]};
}

// The value rows of a masked tile, one a thread of the row tile's 128: rows that nobody attends to become zeros, and
// values that are not finite too, their dimensions noted.  True if this thread's row has a note.
// The other row tile of a pair may do the same at the same time.  A note is written before anything is
// cleared, and read after the values: who finds a value cleared finds the note, so that every note is whole.
__device__ __forceinline__ bool clear_values(const Item &x, int j, uint8_t *stage, Poison *notes, int load)
{
    const int t = threadIdx.x & 127, i = j * kTilePages + t / kPage, slot = t % kPage;
    uint8_t *row = stage + t / kPage * kStageBytes + kTileBytes;
    const bool outside = i >= x.count || x.page(i) * kPage + slot > x.p0 + x.n - 1;
    bool noted = false;
    if (outside) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4 *>(row + swz(slot, c)) = make_uint4(0, 0, 0, 0);
    } else {
        uint32_t hit = 0;  // an exponent of ones carries into the sign's place
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint4 v = *reinterpret_cast<const uint4 *>(row + swz(slot, c));
            hit |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                   ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
        }
        volatile Poison *note = &notes[t];
        uint32_t lo = 0, hi = 0;
        if (hit & 0x80008000u)
            for (int d = 0; d < kD; ++d)
                if ((*reinterpret_cast<volatile uint16_t *>(row + swz(slot, d / 8) + d % 8 * 2) & 0x7f80u) == 0x7f80u)
                    (d < 32 ? lo : hi) |= 1u << (d & 31);
        __threadfence_block();
        if (note->load == load) {
            lo |= note->lo;
            hi |= note->hi;
        }
        noted = (lo | hi) != 0;
        if (hit & 0x80008000u) {
            note->lo = lo;
            note->hi = hi;
            __threadfence_block();
            note->load = load;
            __threadfence_block();
            for (int d = 0; d < kD; ++d)
                if ((d < 32 ? lo : hi) >> (d & 31) & 1u)
                    *reinterpret_cast<volatile uint16_t *>(row + swz(slot, d / 8) + d % 8 * 2) = 0;
        }
    }
    fence_proxy_async_smem();
    return noted;
}

// Half a key tile's scores of one query row become weights, in place (P is the first half of S's columns).  The
// reference m is the row's first scores' maximum (see kMostWeight); -inf: nothing attended to so far.
template <class Mask, class Scale>
__device__ __forceinline__ bool softmax_half(uint32_t ts, uint32_t to, uint32_t tl, const Scale &sc, const Mask &mask, int before,
                                             uint64_t *o_step, volatile int *stop, float &m, float &l)
{
    if (__any_sync(kFull, m == -INFINITY)) {
        const float top = first_reference(ts, sc, mask);
        if (m == -INFINITY)
            m = top;
    }
    uint32_t p0[16], p1[16];
    float s = make_weights(ts, 0, sc, mask, m, p0) + make_weights(ts, 1, sc, mask, m, p1);
    const bool move = !(s < kMostWeight);
    if (__any_sync(kFull, move)) {
        const float top = fmaxf(max_score(ts, 0, sc, mask), max_score(ts, 1, sc, mask));
        const float mn = move ? fmaxf(top, m) : m;
        const float f = move ? ex2_approx(m - mn) : 1.f;
        m = mn;
        l *= f;
        s = make_weights(ts, 0, sc, mask, m, p0) + make_weights(ts, 1, sc, mask, m, p1);
        // Once the product before this one is done, nothing else touches O.  (These scores came
        // after the product before that, so the wait is one phase behind at most.)
        if (!tc::wait_warp(o_step, (before - 1) & 1, stop))
            return false;
        tc::fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t o[16];
            tc::ld16(to + k * 16, o);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tc::st16(to + k * 16, o);
        }
        if constexpr (!Scale::kSum) {
            uint32_t x[16];
            tc::ld16(tl, x);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
            tc::st16(tl, x);
        }
    }
    l += s;
    tc::st16(ts, p0);  // columns 2i, 2i + 1 of S are column i of P
    tc::st16(ts + 16, p1);
    tc::wait_st();
    return true;
}

// Where the partials of part i of an item lie: rows of row tile s.
__device__ __forceinline__ size_t part_rows(const Item &x, int i, int s)
{
    return ((size_t)((x.first + i) * 2 + (i == 0 ? 1 : 0)) * 2 + s) * kRowTile;
}

__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }

// Softmax warps of row tile s: thread = query row (token r / 4 of the tile, head r % 4).
template <bool FP8>
struct Softmax {
    const ChunkArgs &a;
    ChunkShared &sh;
    uint8_t *stages;
    int s, warp, lane, r;
    uint32_t ts, to, tq, tl;
    int loaded = 0, done = 0, used = 0;
    bool queried = false;  // the current item's queries are in tensor memory
    int met[2] = {0, 0};   // times the row tile's warps, and all eight, have met

    __device__ __forceinline__ Softmax(const ChunkArgs &a_, ChunkShared &sh_, uint8_t *stages_, uint32_t tmem)
        : a(a_), sh(sh_), stages(stages_), warp(threadIdx.x >> 5), lane(threadIdx.x & 31)
    {
        s = warp >> 2;
        r = (warp & 3) * 32 + lane;
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        ts = at + kColS + s * 128;
        to = at + kColO + s * 64;
        tq = at + kColQ + s * 32;
        tl = at + kColL + s * 16;
    }

    // The warps of the row tile (all: of both) wait for each other; false if that gave up.
    __device__ __forceinline__ bool meet(bool all)
    {
        uint64_t *bar = &sh.group[all ? 2 : s];
        __syncwarp();
        if (lane == 0)
            tc::mbar_arrive(bar);
        return tc::wait_warp(bar, met[all]++ & 1, &sh.stop);
    }

    // Ticket of a cut item, whose partials all threads of the group have written: `last` for the group that
    // finishes last and has everybody's partials to read.
    __device__ __forceinline__ bool draw_ticket(const Item &x, bool all, bool &last)
    {
        const int row_tile = all ? 0 : s;
        __threadfence();
        if (!meet(all))
            return false;
        int *flag = &sh.last[all ? 2 : s];
        if ((int)threadIdx.x == row_tile * 128) {
            int *ticket = &a.tickets[x.first * 2 + row_tile];
            int drawn;
            asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(drawn) : "l"(ticket) : "memory");
            sh.taken[x.me == 0][row_tile] = 1;
            *flag = drawn == x.parts - 1;
            if (drawn == x.parts - 1)
                *ticket = 0;
        }
        if (!meet(all))
            return false;
        last = *(volatile int *)flag != 0;
        if (last)
            __threadfence();
        return true;
    }

    __device__ __forceinline__ size_t row_at(const Item &x) const
    {
        return ((size_t)(x.t0 + x.token(s) + r / kGroup) * kHq + x.head(s) * kGroup + r % kGroup) * kD;
    }

    // An item's query rows into tensor memory: 64 values, two to a column.  (Every product of the
    // previous item with its queries is done when its last scores are there.)
    __device__ __forceinline__ void queries(const Item &x)
    {
        const bool live = r / kGroup < x.tokens(s);
        uint32_t w[32];
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + row_at(x));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4 v = live ? src[i] : make_uint4(0, 0, 0, 0);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
        tc::st32(tq, w);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0)
            tc::mbar_arrive(&sh.q_full[s]);
    }

    // A piece of row tiles; false if a wait gave up.
    __device__ __forceinline__ bool tiles_piece(Feed &feed, const Item &x)
    {
        if (!queried)
            queries(x);
        queried = false;
        const int live = x.tokens(s), nt = x.j1 - x.j0;
        const bool idle = (warp & 3) * 8 >= live;  // no row of the warp is a query: it only keeps step
        const int pos = x.p0 + x.token(s) + min(r / kGroup, live - 1);
        float m = -INFINITY, l = 0.f;
        int bad = 0;
        uint32_t nan_lo = 0, nan_hi = 0;
        for (int j = 0; j < nt; ++j) {
            const int seq = loaded + x.order(s, j), st = seq % kStages;
            const bool masked = x.masked(x.j0 + j, a.window);
            if (a.expire && s == 0 && used == 0 && j == 0 && blockIdx.x == 0) {
                *(volatile int *)&sh.stop = 1;
                return false;
            }
            if (FP8 || masked)  // what this thread reads of the stage itself
                if (!tc::wait_warp(&sh.full[st], (seq / kStages) & 1, &sh.stop))
                    return false;
            bool noted = false;
            if (masked) {
                if (clear_values(x, x.j0 + j, stages + st * kStageSize, sh.poison[st], seq))
                    sh.noted[s] = seq;
                if (!meet(false))
                    return false;
                noted = *(volatile int *)&sh.noted[s] == seq;
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                if (!tc::wait_warp(&sh.s_full[s][hf], (done + j) & 1, &sh.stop))
                    return false;
                if (!idle) {
                    tc::fence_after();
                    const int before = 2 * (done + j) + hf;  // products of this row tile so far
                    const auto half = [&](const auto &sc) {
                        uint64_t *step = &sh.o_step[s];
                        if (!masked)
                            return softmax_half(ts + hf * kHalf, to, tl, sc, EveryColumn{}, before, step, &sh.stop, m, l);
                        const ColumnBits mask = columns(x, x.j0 + j, hf, pos, a.window, a.sinks);
                        if (noted) {
                            for (int i = 0; i < kHalf; ++i)
                                if ((i < 32 ? mask.w0 : mask.w1) >> (i & 31) & 1u) {
                                    const Poison &note = sh.poison[st][i / 8 * kPage + 8 * hf + i % 8];
                                    if (note.load == seq) {
                                        nan_lo |= note.lo;
                                        nan_hi |= note.hi;
                                    }
                                }
                        }
                        return softmax_half(ts + hf * kHalf, to, tl, sc, mask, before, step, &sh.stop, m, l);
                    };
                    bool go;
                    if constexpr (FP8) {
                        const float2 *sc = reinterpret_cast<const float2 *>(sh.scales[st]) + hf * 32;
                        go = half(RowScales{sc, sc + 64, sc + 128});
                    } else {
                        go = half(OneFactor{a.scale_log2});
                    }
                    if (!go)
                        return false;
                    if (hf == 0)
                        bad |= *(volatile int *)&sh.bad[st];
                    tc::fence_before();
                }
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(&sh.p_full[s][hf]);
            }
        }
        // the next item's first scores are made while this one's last product and its output end
        const Item *y = feed.look(1);
        if (y && y->kind != plan::kSingle) {
            queries(*y);
            queried = true;
        }
        if (!tc::wait_warp(&sh.o_full[s], used & 1, &sh.stop))
            return false;
        tc::fence_after();
        if constexpr (!FP8) {
            uint32_t sums[16];
            tc::ld16(tl, sums);
            l = __uint_as_float(sums[0]);
        }
        if (bad && r == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
        const bool mine = r / kGroup < live;
        uint32_t o[2][32];
        tc::ld32(to, o[0]);
        tc::ld32(to + 32, o[1]);
        if (nan_lo | nan_hi) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if (nan_lo >> i & 1u)
                    o[0][i] = 0x7fffffffu;
                if (nan_hi >> i & 1u)
                    o[1][i] = 0x7fffffffu;
            }
        }
        if (x.parts == 1) {
            if (mine)
                store_row(x, reinterpret_cast<const float *>(o[0]), bad ? 0.f : inverse_sum(l), bad);
        } else {
            const size_t at = part_rows(x, x.me, s) + r;
            if (mine) {
                float4 *to4 = reinterpret_cast<float4 *>(a.part_o + at * kD);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t *v = &o[i / 8][i % 8 * 4];
                    __stcg(to4 + i, make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]),
                                                __uint_as_float(v[3])));
                }
                __stcg(a.part_ml + at, make_float2(bad ? INFINITY : m, l));
            }
            bool last;
            if (!draw_ticket(x, false, last))
                return false;
            if (last && mine)
                join(x);
        }
        loaded += x.loads();
        done += nt;
        ++used;
        return true;
    }

    __device__ __forceinline__ void store_row(const Item &x, const float *o, float f, bool bad) const
    {
        uint4 *dst = reinterpret_cast<uint4 *>(a.out + row_at(x));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint4 v = make_uint4(pack_bf16x2(o[8 * i] * f, o[8 * i + 1] * f), pack_bf16x2(o[8 * i + 2] * f, o[8 * i + 3] * f),
                                 pack_bf16x2(o[8 * i + 4] * f, o[8 * i + 5] * f),
                                 pack_bf16x2(o[8 * i + 6] * f, o[8 * i + 7] * f));
            dst[i] = bad ? make_uint4(0, 0, 0, 0) : v;
        }
    }

    // This thread's row of a cut item, of all parts.
    __device__ __forceinline__ void join(const Item &x) const
    {
        float M = -INFINITY;
        for (int i = 0; i < x.parts; ++i)
            M = fmaxf(M, __ldcg(a.part_ml + part_rows(x, i, s) + r).x);
        float o[kD], l = 0.f;
#pragma unroll
        for (int i = 0; i < kD; ++i)
            o[i] = 0.f;
        for (int i = 0; i < x.parts; ++i) {
            const size_t at = part_rows(x, i, s) + r;
            const float2 ml = __ldcg(a.part_ml + at);
            const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
            if (ml.x == -INFINITY)
                continue;
            l = fmaf(f, ml.y, l);
            const float4 *src = reinterpret_cast<const float4 *>(a.part_o + at * kD);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const float4 v = __ldcg(src + c);
                o[4 * c] = fmaf(f, v.x, o[4 * c]);
                o[4 * c + 1] = fmaf(f, v.y, o[4 * c + 1]);
                o[4 * c + 2] = fmaf(f, v.z, o[4 * c + 2]);
                o[4 * c + 3] = fmaf(f, v.w, o[4 * c + 3]);
            }
        }
        store_row(x, o, inverse_sum(l), M == INFINITY);
    }

    // ---- a single token: the 8 warps take a page each of every key tile

    __device__ __forceinline__ bool single_piece(const Item &x)
    {
        std::conditional_t<FP8, fp8::Fp8MmaWarp, MmaWarp> w;
        const uint16_t *q = a.q + ((size_t)x.t0 * kHq + x.g * kGroup) * kD;
        if constexpr (FP8)
            w.init(q, a.scale_log2, lane);
        else
            w.init(q, a.scale_log2, lane, nullptr);
        constexpr int kUnit = FP8 ? kFp8Unit : kStageBytes;
        const int p = x.p0, lo = a.window ? max(p + 1 - a.window, 0) : 0;
        int bad = 0;
        for (int j = x.j0; j < x.j1; ++j) {
            const int seq = loaded + j - x.j0, st = seq % kStages;
            if (a.expire && used == 0 && seq == 0 && blockIdx.x == 0) {
                *(volatile int *)&sh.stop = 1;
                return false;
            }
            if (!tc::wait_warp(&sh.full[st], (seq / kStages) & 1, &sh.stop))
                return false;
            bad |= *(volatile int *)&sh.bad[st];
            const int i = j * kTilePages + warp;
            if (i < x.count) {
                const uint8_t *page = stages + st * kStageSize + warp * kUnit;
                const int first = x.page(i) * kPage;
                const uint32_t upto = p + 1 - first >= kPage ? 0xffffu : (1u << (p + 1 - first)) - 1;
                const uint32_t below = (1u << min(max(lo - first, 0), kPage)) - 1;
                const uint32_t sunk = (1u << min(max(a.sinks - first, 0), kPage)) - 1;
                const uint32_t bits = upto & (~below | sunk);
                if (bits == 0xffffu)
                    w.page(page, EveryToken{});
                else if (bits)
                    w.page(page, TokenSet{bits});
            }
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(&sh.empty[st]);
        }
        w.store_state(sh.states[warp]);
        if (!meet(true))
            return false;
        const int hl = threadIdx.x >> 6, d = threadIdx.x & 63;
        float M = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
        for (int i = 0; i < kTeam; ++i)
            M = fmaxf(M, sh.states[i][hl]);
#pragma unroll
        for (int i = 0; i < kTeam; ++i) {
            const float mi = sh.states[i][hl], f = mi == -INFINITY ? 0.f : ex2_approx(mi - M);
            l = fmaf(f, sh.states[i][4 + hl], l);
            o = fmaf(f, sh.states[i][8 + hl * kD + d], o);
        }
        if (!meet(true))  // the states may be written again
            return false;
        if (bad && threadIdx.x == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
        bool write = x.parts == 1;
        if (!write) {
            const size_t at = part_rows(x, x.me, 0) + hl;
            __stcg(a.part_o + at * kD + d, o);
            if (d == 0)
                __stcg(a.part_ml + at, make_float2(bad ? INFINITY : M, l));
            if (!draw_ticket(x, true, write))
                return false;
            if (write) {
                M = -INFINITY;
                for (int i = 0; i < x.parts; ++i)
                    M = fmaxf(M, __ldcg(a.part_ml + part_rows(x, i, 0) + hl).x);
                bad = M == INFINITY;
                l = o = 0.f;
#pragma unroll 4
                for (int i = 0; i < x.parts; ++i) {
                    const size_t from = part_rows(x, i, 0) + hl;
                    const float2 ml = __ldcg(a.part_ml + from);
                    const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
                    l = fmaf(f, ml.y, l);
                    o = fmaf(f, __ldcg(a.part_o + from * kD + d), o);
                }
            }
        }
        if (write) {
            const __nv_bfloat16 v = __float2bfloat16_rn(bad ? 0.f : o * inverse_sum(l));
            a.out[((size_t)x.t0 * kHq + x.g * kGroup + hl) * kD + d] = *reinterpret_cast<const uint16_t *>(&v);
        }
        loaded += x.j1 - x.j0;
        return true;
    }

    __device__ __forceinline__ void run()
    {
        Feed feed(sh);
        for (const Item *x; (x = feed.look()) != nullptr; feed.let_go())
            if (!(x->kind == plan::kSingle ? single_piece(*x) : tiles_piece(feed, *x)))
                return;
    }
};

// ------------------------------------------------------------------ the kernel

template <bool FP8>
__global__ void __launch_bounds__(chunk_threads(FP8), 1)
chunk_kernel(const __grid_constant__ CUtensorMap tmap, ChunkArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded address: the compiler keeps shared-memory instructions)
    uint8_t *stages = smem_raw + (-smem_addr(smem_raw) & 1023u);
    uint8_t *raws = stages + kStages * kStageSize;  // (BF16 pages: the ones)
    ChunkShared &sh = *reinterpret_cast<ChunkShared *>(raws + (FP8 ? kRaws * kRawSize : kOnesSize));
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], FP8 ? kConverters : 1);
            mbar_init(&sh.empty[i], kTeam);
        }
        for (int i = 0; i < kRaws; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], kConverters);
        }
        for (int s = 0; s < 2; ++s) {
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sh.s_full[s][h], 1);
                mbar_init(&sh.p_full[s][h], 4);
            }
            mbar_init(&sh.q_full[s], 4);
            mbar_init(&sh.o_step[s], 1);
            mbar_init(&sh.o_full[s], 1);
            mbar_init(&sh.drained[s], 1);
            mbar_init(&sh.group[s], 4);
            sh.noted[s] = -1;
        }
        mbar_init(&sh.group[2], kTeam);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], consumers(FP8));
        }
        sh.stop = 0;
        sh.taken[0][0] = sh.taken[0][1] = sh.taken[1][0] = sh.taken[1][1] = 0;
        fence_barrier_init();
    }
    if (warp == kIssuer)
        tc::alloc<kCols>(&sh.tmem);
    for (int i = threadIdx.x; i < kStages * kTilePages * kPage; i += chunk_threads(FP8))
        (&sh.poison[0][0])[i].load = -1;
    if (!FP8) {
        for (int i = threadIdx.x; i < kOnesSize / 4; i += chunk_threads(FP8))
            reinterpret_cast<uint32_t *>(raws)[i] = 0x3f803f80u;
        fence_proxy_async_smem();
    }
    grid_dependency_wait();
    allow_dependent_launch();
    make_plan<FP8>(a, sh);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sh.tmem;
    // FP8: 512 threads of 128 registers; the softmax warps take 168, so that none spill, and leave the
    // others 88.  (Registers move by fours of warps.)
    if (warp < kLoader) {
        if constexpr (FP8)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        Softmax<FP8>(a, sh, stages, tmem).run();
    } else {
        if constexpr (FP8)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == kLoader)
            loader<FP8>(&tmap, a, stages, raws, sh);
        else if (warp < kIssuer + 2)
            issuer<FP8>(stages, raws, sh, tmem, warp - kIssuer);
        else if (warp == kScheduler)
            scheduler<FP8>(a, sh);
        else if (FP8)
            converter(a, raws, stages, sh);
    }
    __syncthreads();
    if (sh.stop && warp == kScheduler) {
        // the tickets that were not drawn, so that the next call finds zeros
        for_each_piece<FP8>(a, sh, [&](const Item &x) {
            const int which = x.me == 0;
            if (x.parts > 1 && (threadIdx.x & 31) == 0)
                for (int s = 0; s < (x.kind == plan::kSingle ? 1 : 2); ++s)
                    if (!sh.taken[which][s] && atomicAdd(&a.tickets[x.first * 2 + s], 1) == x.parts - 1)
                        a.tickets[x.first * 2 + s] = 0;
            return true;
        });
        if ((threadIdx.x & 31) == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_TIMEOUT);
    }
    if (warp == kIssuer)
        tc::dealloc<kCols>(tmem);
}

struct ChunkWorkspace {
    size_t tickets, ml, o;
    size_t total() const { return tickets + ml + o; }
};

ChunkWorkspace chunk_workspace()
{
    ChunkWorkspace w;
    w.tickets = align256((size_t)kSms * 2 * sizeof(int));
    w.ml = align256((size_t)kSms * 4 * kRowTile * sizeof(float2));
    w.o = (size_t)kSms * 4 * kRowTile * kD * sizeof(float);
    return w;
}

template <bool FP8>
int launch_chunk(const pkv_pool *pool, const ChunkArgs &a, cudaStream_t s, bool pdl)
{
    const CUtensorMap *tmap = pool_tensor_map(pool);
    if (!tmap)
        return PKV_ERR_CUDA;
    constexpr int smem = 1024 + kStages * kStageSize + (FP8 ? kRaws * kRawSize : kOnesSize) + (int)sizeof(ChunkShared);
    static_assert(smem <= 227 * 1024, "shared memory of an SM");
    static PerDeviceOnce attr;
    if (const int st = ensure_smem_attr(attr, chunk_kernel<FP8>, smem); st != PKV_OK)
        return st;
    return launch_kernel(chunk_kernel<FP8>, dim3(kSms), dim3(chunk_threads(FP8)), smem, s, pdl, *tmap, a);
}

bool chunk_args_ok(int B, int T) { return B >= 1 && B <= kMaxRows && T >= 1 && T <= INT32_MAX / 16; }

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_chunk_attention_workspace_bytes(int B, int T)
{
    return pkv::chunk_args_ok(B, T) ? pkv::chunk_workspace().total() : 0;
}

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
    const ChunkWorkspace ws = chunk_workspace();
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
    a.tickets = static_cast<int *>(workspace);
    a.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + ws.tickets);
    a.part_o = reinterpret_cast<float *>(static_cast<char *>(workspace) + ws.tickets + ws.ml);
    a.expire = (options & PKV_STEP_TEST_EXPIRE_WAIT) ? 1 : 0;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    const bool pdl = !(options & PKV_STEP_NO_PDL);
    return pool->kv_format == PKV_KV_FP8 ? launch_chunk<true>(pool, a, s, pdl) : launch_chunk<false>(pool, a, s, pdl);
}
