// pkv_chunk.cu -- causal attention of a step's new tokens over their sequences' pages.
//
//     out[t][h] = sum_j softmax_j(scale * q[t][h] . K_j) V_j,   j <= p(t), and j > p(t) - window or j < sinks.
//
// 32 tokens and the 4 query heads of a KV head are 128 rows that meet the same keys: S = Q K^T and O += P V
// on the tensor cores (tcgen05), Q, S, P and O in tensor memory, K and V in shared memory as TMA brought the
// pages.  A CTA has two such row tiles at a time, each with four softmax warps (a thread a row) and an issuer
// warp, so that one's products fill the other's exponentials.  Sequences that bring a single token, 4 rows a KV
// head, are mostly left to a kernel of their own (pkv_chunk_single.cu; apart_of()).  pkv_chunk_plan.cuh says
// how the work is cut into one run for every CTA.
//
// Masks: only tiles in which some row does not attend to some token (the last ones, and a window's
// first) are masked, by 64 bits a row and half tile.  A weight of 0 times a value that is not finite would
// not be 0, so in those tiles an issuer warp (FP8: the warps that convert) looks for such values and clears them; rows
// that attend to one get NaN in its dimension at the end.  (By the softmax warps themselves: 16 prompts of 2048 305 us
// where 259 were without.)
//
// What bounds it is the way from a half tile's scores to its weights and back: 2048 tokens behind 14000 take 228 us (1110
// TFLOP/s, where a large product does 1964), with the tensor pipe and the special-function pipe half busy each; FP8
// pages, whose codes are converted and whose scales go to scores and weights, 339.  16 prompts of 2048 200, FP8 371.  (The
// comparisons below were each taken in turn, when the choice was made: 16 prompts then took 194 to 260.)
#include <cmath>

#include "pkv_chunk_run.cuh"
#include "pkv_tiles.cuh"

namespace pkv {
namespace chunk {
namespace {

using namespace tiles;

constexpr int kStages = 4, kRaws = 2;
constexpr int kLoader = 8, kIssuer = 9, kScheduler = 11, kPreparer = 12;   // warps: 2 x 4 softmax, ...
constexpr int kPreparers = 4;
constexpr int kRowBytes = 128 + 16;  // a query or output row in shared memory, padded to other banks
constexpr int kRowsSize = 2 * kRowTile * kRowBytes;
// What the weights are multiplied with for their sums, 16 columns of 64 places: ones; FP8: for every stage and half
// the inverses of V's scales, as two BF16 numbers in the first two columns (the others do not matter).
constexpr int sums_size(bool fp8) { return fp8 ? (2 * kStages + 1) * 1024 : 2048; }
constexpr int kCols = 512;           // tensor memory, all of it
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384, kColL = 448;  // + 128 / 64 / 32 / 16 for the second row tile

template <bool FP8>
struct TileRun {
    static constexpr int kThreads = (FP8 ? kPreparer + kPreparers : kPreparer) * 32;
    static constexpr int kConsumers = FP8 ? 8 + 3 + kPreparers : 8 + 3;
    static constexpr bool kSingles = false;
    // Of a CTA's run (64 tokens behind 2000 23 us, 200 behind 500 21; at 64 eighths 25 and 30, at 16 24 and 21).
    static constexpr int kLeast = 32;
    // in eighths of the time of a BF16 key tile of two row tiles; what an item costs besides: 24 (18: 16 prompts of 2048
    // 203 us, 30: 194, where this takes 196, but 33 tokens behind 500, cut then, 18 where 15), FP8 38 (30: 395, this 381)
    static __device__ __forceinline__ Costs costs()
    {
        return FP8 ? Costs{{0, 14, 16, 0}, {0, 38, 38, 0}} : Costs{{0, 8, 9, 0}, {0, 24, 24, 0}};
    }
};

// A value row of a masked tile that holds something not finite: the load it belongs to, and which dimensions.
struct Poison {
    int load;
    uint32_t lo, hi;
};

struct ChunkShared : RunShared {
    uint64_t full[kStages], empty[kStages];      // a stage holds its pages / has been read by all
    uint64_t raw_full[kRaws], raw_empty[kRaws];  // the same of the raw units
    uint64_t s_full[2][2], p_full[2][2];         // [row tile][half]: scores are in tensor memory / weights are
    uint64_t o_step[2];                          // one more product of weights and values is done
    uint64_t q_full[2], o_full[2];               // once an item: the queries are in / its last product is done
    uint64_t checked[kStages];                   // (BF16) the values of a masked load have been gone through
    uint64_t group[3];                           // row tile s's warps (2: the preparers) have come so far
    uint64_t drained[2];
    uint32_t tmem;
    int bad[kStages], raw_bad[kRaws];            // the tile has a bad page id
    int noted[kStages];                          // the last load into the stage with notes on values (see Poison)
    int claimed;                                 // (BF16) pairs' masked loads up to here are being gone through
    int last[2];                                 // row tile s: this CTA finished the item last
    Poison poison[kStages][kTilePages * kPage];
    int64_t sums[(kPreparer + kPreparers) * 32];
    alignas(16) float scales[kStages][2][kTilePages * kPage];  // (FP8) row scales: K's times scale log2 e, V's
};

// A stage is free after two arrivals: those of both row tiles' last products, or of one and one that whoever fills the
// stage gives in advance.
__device__ __forceinline__ bool given_in_advance(int kind) { return kind != plan::kPair; }

// ------------------------------------------------------------------ loader

// The pages of every piece's key tiles into the ring of stages (FP8: of raw units).  A tile that the pages do not fill
// repeats the last one (its places are masked); a bad page id is replaced by page 0 and the tile marked.
template <bool FP8>
__device__ __forceinline__ void loader(const CUtensorMap *tmap, const ChunkArgs &a, uint8_t *stages, uint8_t *raws,
                                       ChunkShared &sh)
{
    constexpr int kRing = FP8 ? kRaws : kStages, kSize = FP8 ? kRawSize : kStageSize;
    uint64_t *full = FP8 ? sh.raw_full : sh.full, *empty = FP8 ? sh.raw_empty : sh.empty;
    int *marks = FP8 ? sh.raw_bad : sh.bad;
    uint8_t *ring = FP8 ? raws : stages;
    const int lane = threadIdx.x & 31;
    uint64_t policy;  // pages are read by several CTAs: no eviction hint
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    Feed feed(sh);
    int seq = 0;                 // key tiles loaded so far
    int ahead = -1, first4 = 0;  // the item whose first ids are there
    bool go = true;
    for (const Item *p; go && (p = feed.look()) != nullptr; feed.let_go()) {
        const Item x = *p;
        const int heads = x.kind == plan::kHeads ? 2 : 1;
        // lane l: the id of page l of the current run of 4 key tiles, and of the next run: their loads are a run ahead
        const auto ids_of = [&](const Item &y, int j) {
            return (a.bt + (size_t)y.b * a.max_blocks)[y.page(min(j * kTilePages + lane, y.count - 1))];
        };
        int id4 = 0, next4 = ahead == feed.n ? first4 : ids_of(x, x.j0);
        unsigned bad4 = 0;
        for (int j = x.j0; j < x.j1 && go; ++j) {
            const int in4 = (j - x.j0) & 3;
            if (in4 == 0) {
                id4 = next4;
                if (j + 4 < x.j1) {
                    next4 = ids_of(x, j + 4);
                } else if (const Item *y = feed.look(1)) {  // (of the next item: it is there long before)
                    first4 = ids_of(*y, y->j0);
                    ahead = feed.n + 1;
                }
                const bool out = id4 < 0 || id4 >= a.num_pages;
                bad4 = __ballot_sync(kFull, out);
                if (out)
                    id4 = 0;
            }
            const int id = __shfl_sync(kFull, id4, in4 * kTilePages + lane % kTilePages);
            const int bad = (bad4 >> (in4 * kTilePages)) & ((1u << kTilePages) - 1);
            for (int h = 0; h < heads; ++h) {
                const int st = seq % kRing;
                if (seq >= kRing && !wait_for(&empty[st], (seq / kRing - 1) & 1, &sh.stop)) {
                    go = false;
                    break;
                }
                fence_proxy_async_smem();  // (the place's readers and writers so far may be threads)
                uint8_t *dst = ring + st * kSize;
                if (lane == 0) {
                    marks[st] = bad;
                    if (!FP8 && given_in_advance(x.kind))
                        tc::mbar_arrive(&empty[st]);
                    mbar_arrive_expect_tx(&full[st], kSize);
                }
                __syncwarp();
                if (lane < kTilePages) {
                    if (FP8)
                        fp8::tma_load_unit(dst + lane * kFp8Unit, tmap, &full[st], x.g + h, id, policy);
                    else
                        tma_load_page_head(dst + lane * kStageBytes, tmap, &full[st], x.g + h, id, policy);
                }
                ++seq;
            }
        }
    }
    if (*(volatile int *)&sh.stop)  // let the copies in flight land (bounded)
        for (int i = max(seq - kRing, 0); i < seq; ++i)
            (void)mbar_wait_warp(&full[i % kRing], (i / kRing) & 1);
}

// ------------------------------------------------------------------ values of masked tiles

// The value rows of a masked tile by THREADS threads (`t` of them): a weight of 0 times a value that is not finite would
// not be 0, so such values become zeros, and where somebody may attend to them their dimensions are noted.
template <int THREADS>
__device__ __forceinline__ void check_values(const Item &x, int j, uint8_t *stage, Poison *notes, int *noted, int load, int t)
{
#pragma unroll 1
    for (int key = t; key < kTilePages * kPage; key += THREADS) {
        const int i = j * kTilePages + key / kPage, slot = key % kPage;
        uint8_t *row = stage + key / kPage * kStageBytes + kTileBytes;
        uint32_t hit = 0;  // an exponent of ones carries into the sign's place
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint4 v = *reinterpret_cast<const uint4 *>(row + swz(slot, c));
            hit |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                   ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
        }
        if (!(hit & 0x80008000u))
            continue;
        uint32_t lo = 0, hi = 0;
        for (int d = 0; d < kD; ++d) {
            uint16_t *v = reinterpret_cast<uint16_t *>(row + swz(slot, d / 8)) + d % 8;
            if ((*v & 0x7f80u) == 0x7f80u) {
                (d < 32 ? lo : hi) |= 1u << (d & 31);
                *v = 0;
            }
        }
        if (i < x.count && x.page(i) * kPage + slot < x.p0 + x.n) {  // (what is behind the last token reaches nobody)
            notes[key] = {load, lo, hi};
            *noted = load;
        }
        fence_proxy_async_smem();
    }
}

// ------------------------------------------------------------------ preparers (FP8 row tiles; 128 threads)

// Units become BF16 values, and masked tiles are gone through.
__device__ __forceinline__ void preparer(const ChunkArgs &a, const uint8_t *raws, uint8_t *stages, uint8_t *sums, ChunkShared &sh)
{
    const int t = threadIdx.x - kPreparer * 32, lane = threadIdx.x & 31;
    Feed feed(sh);
    int seq = 0, checks = 0;
    for (const Item *p; (p = feed.look()) != nullptr; feed.let_go()) {
        const Item x = *p;
        const int n = x.loads();
        for (int i = 0; i < n; ++i, ++seq) {
            const int j = x.j0 + (x.kind == plan::kHeads ? i / 2 : i), rs = seq % kRaws, st = seq % kStages;
            if (!wait_for(&sh.raw_full[rs], (seq / kRaws) & 1, &sh.stop) ||
                (seq >= kStages && !wait_for(&sh.empty[st], (seq / kStages - 1) & 1, &sh.stop)))
                return;
            const uint8_t *raw_tile = raws + rs * kRawSize;
            uint8_t *stage = stages + st * kStageSize;
            convert_codes(raw_tile, stage, t);
            {  // row scales in the order of the scores' columns; thread = (page, slot)
                const int page = t / kPage, slot = t % kPage, at = page * 8 + slot % 8;
                const float *row = reinterpret_cast<const float *>(raw_tile + page * kFp8Unit + kFp8UnitCodes);
                const float f = row[kPage + slot];
                // (a scale below 2^-100, of rows of nothing, as 2^-100: weights are counted by its inverse;
                // one that is not finite counts nothing: rows that attend to it are not finite by P)
                const float v = fabsf(f) < 0x1p-100f ? 0x1p-100f : f;
                const float inv = fabsf(v) < INFINITY ? __frcp_rn(v) : 0.f;
                sh.scales[st][0][slot / 8 * kHalf + at] = row[slot] * a.scale_log2;
                sh.scales[st][1][slot / 8 * kHalf + at] = v;
                uint8_t *sum = sums + (st * 2 + slot / 8) * 1024 + slot % 8 * 2;
                const __nv_bfloat16 hi = __float2bfloat16_rn(inv), lo = __float2bfloat16_rn(inv - __bfloat162float(hi));
                *reinterpret_cast<__nv_bfloat16 *>(sum + page * 16) = hi;  // (row 0, row 1 of the swizzled operand)
                *reinterpret_cast<__nv_bfloat16 *>(sum + 128 + (page ^ 1) * 16) = lo;
            }
            if (t == 0) {
                sh.bad[st] = sh.raw_bad[rs];
                if (given_in_advance(x.kind))
                    tc::mbar_arrive(&sh.empty[st]);
            }
            if (x.masked(j)) {  // (rows that other warps have written)
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(&sh.group[2]);
                if (!wait_for(&sh.group[2], checks++ & 1, &sh.stop))
                    return;
                check_values<kPreparers * 32>(x, j, stage, sh.poison[st], &sh.noted[st], seq, t);
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
__device__ __forceinline__ void issuer(uint8_t *stages, const uint8_t *sums, ChunkShared &sh, uint32_t tmem, int s)
{
    const uint32_t base = smem_addr(stages), sum0 = smem_addr(sums), tl = tmem + kColL + s * 16;
    const uint32_t ts = tmem + kColS + s * 128, to = tmem + kColO + s * 64, tq = tmem + kColQ + s * 32;
    Feed feed(sh);
    // loads of earlier pieces, those of masked tiles, key tiles of this row tile, pieces with row tiles
    int loaded = 0, checks = 0, done = 0, used = 0;
    for (const Item *p; (p = feed.look()) != nullptr; feed.let_go()) {
        const Item x = *p;
        const int nt = x.j1 - x.j0;
        const auto scores = [&](int j, int h) {
            const int seq = loaded + x.order(s, j), st = seq % kStages;
            if (h == 0) {
                if (!wait_for(&sh.full[st], (seq / kStages) & 1, &sh.stop))
                    return false;
                tc::fence_after();
            }
            issue_scores(base + st * kStageSize + h * 1024, ts + h * kHalf, tq, &sh.s_full[s][h]);
            return true;
        };
        const auto first_at = [&](int check) {
            int before = 0;
            if ((threadIdx.x & 31) == 0)
                before = atomicMax(&sh.claimed, check + 1);
            return __shfl_sync(kFull, before, 0) <= check;
        };
        const auto output = [&](int j, int h) {
            const int seq = loaded + x.order(s, j), st = seq % kStages;
            if (!FP8 && h == 0 && x.masked(x.j0 + j)) {
                // (a pair's values, which both row tiles read, by the issuer that comes first; by the first row tile's,
                // the second waited for it up to 6500 clocks an item)
                const int check = checks + x.masked_loads(j) + (x.kind == plan::kHeads ? s : 0);
                uint64_t *checked = &sh.checked[check % kStages];
                if (x.kind == plan::kHeads || first_at(check)) {
                    check_values<32>(x, x.j0 + j, stages + st * kStageSize, sh.poison[st], &sh.noted[st], seq,
                                     threadIdx.x & 31);
                    __syncwarp();
                    if ((threadIdx.x & 31) == 0)
                        tc::mbar_arrive(checked);
                }
                if (!wait_for(checked, (check / kStages) & 1, &sh.stop))
                    return false;
            }
            if (!wait_for(&sh.p_full[s][h], (done + j) & 1, &sh.stop))
                return false;
            tc::fence_after();
            const uint32_t v = base + st * kStageSize + kTileBytes + h * 1024, pw = ts + h * kHalf;
            uint64_t *empty = h == 1 ? &sh.empty[st] : nullptr;
            uint64_t *last = h == 1 && j + 1 == nt ? &sh.o_full[s] : nullptr;
            const uint32_t sum = sum0 + (FP8 ? (st * 2 + h) * 1024 : 0);
            if (j == 0 && h == 0)
                issue_output<true, true, FP8 ? 2 : 0>(v, to, pw, sum, tl, empty, 1, &sh.o_step[s], last);
            else
                issue_output<false, true, FP8 ? 2 : 0>(v, to, pw, sum, tl, empty, 1, &sh.o_step[s], last);
            return true;
        };
        bool go = wait_for(&sh.q_full[s], used & 1, &sh.stop);
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
        checks += x.masked_loads(nt);
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

// The first columns of a half tile, those of the first t tokens (or fewer than none) from its first column's on, whose
// pages follow one another: 8 columns, then 8 tokens of the other half.
__device__ __forceinline__ uint2 first_columns(int t)
{
    t = min(max(t, 0), 8 * kPage);
    const int n = t / kPage * 8 + min(t % kPage, 8);
    const int lo = min(n, 32), hi = max(n - 32, 0);
    return make_uint2(lo == 32 ? kFull : (1u << lo) - 1, hi == 32 ? kFull : (1u << hi) - 1);
}

// What a row at position p attends to in half hf of key tile j.  (What lies behind the item's last page lies behind p.)
__device__ __forceinline__ uint2 columns(const Item &x, int j, int hf, int p, int window, int sinks)
{
    const int at = j * kTilePages, lo = window ? max(p + 1 - window, 0) : 0;
    if (at >= x.sink || at + kTilePages <= x.sink) {
        const int first = x.page(at) * kPage + 8 * hf;
        uint2 w = first_columns(p + 1 - first);
        if (window) {
            const uint2 below = first_columns(lo - first), sunk = first_columns(sinks - first);
            w.x &= ~below.x | sunk.x;
            w.y &= ~below.y | sunk.y;
        }
        return w;
    }
    uint32_t w[2] = {0, 0};  // (the tile in which the window's pages follow the first ones)
#pragma unroll
    for (int i = 0; i < kTilePages; ++i) {
        const int first = x.page(at + i) * kPage + 8 * hf;
        const uint32_t bits = low_bits(p + 1 - first) & (~low_bits(lo - first) | low_bits(sinks - first));
        w[i / 4] |= bits << (i % 4 * 8);
    }
    return make_uint2(w[0], w[1]);
}

// The dimensions of noted values that a row attends to in half hf of the tile.
__device__ __noinline__ void reached(uint2 mask, const Poison *notes, int hf, int load, uint32_t &lo, uint32_t &hi)
{
    for (int i = 0; i < kHalf; ++i) {
        const Poison &note = notes[i / 8 * kPage + 8 * hf + i % 8];
        if (((i < 32 ? mask.x : mask.y) >> (i & 31) & 1u) && note.load == load) {
            lo |= note.lo;
            hi |= note.hi;
        }
    }
}

// What half a key tile's scores of one query row need besides themselves: the factor of all of them, or (FP8) the row
// scales of the 64 columns, K's (times the factor) and V's; the columns that count; where S, O and the sums are.
struct HalfRow {
    uint32_t ts, to, tl;
    float c;
    const float4 *ks, *vs;
    uint2 mask;
    template <bool MASKED>
    __device__ __forceinline__ void drop(int i, float2 &x, float to_) const  // columns 2 i, 2 i + 1
    {
        if (MASKED) {
            const uint32_t w = i < 16 ? mask.x : mask.y;
            x.x = w & (1u << (2 * i & 31)) ? x.x : to_;
            x.y = w & (2u << (2 * i & 31)) ? x.y : to_;
        }
    }
};

// The maximum of the scores that count, times the factors.
template <bool FP8, bool MASKED>
__device__ __noinline__ float top_score(HalfRow h)
{
    float mx = -INFINITY;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t w[32];
        tc::ld32(h.ts + q * 32, w);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float4 f = FP8 ? h.ks[q * 8 + i / 2] : make_float4(h.c, h.c, h.c, h.c);
            float2 x = tc::mul2(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), make_float2(f.x, f.y));
            float2 y = tc::mul2(make_float2(__uint_as_float(w[2 * i + 2]), __uint_as_float(w[2 * i + 3])), make_float2(f.z, f.w));
            h.drop<MASKED>(q * 16 + i, x, -INFINITY);
            h.drop<MASKED>(q * 16 + i + 1, y, -INFINITY);
            mx = tc::max3(tc::max3(mx, x.x, x.y), y.x, y.y);
        }
    }
    return mx;
}

// How far a reference lies above the maximum that it is taken from, and the weight that moves it.  BF16 pages: 2, which
// one bit of the rounded weights shows (as a maximum over them it took 268 us where this takes 253: 2048 tokens behind
// 14000); so it lies 2^60 above, and weights down to 2^-66 of the first ones' largest count.  (2^32
// above: outliers among the keys move it, 305 us for 16 prompts of 2048 where 239 were.)  FP8 pages: the
// weights are multiplied with V's scales, which may be small, so it lies at the maximum, and 2^64 moves it.
//
// What is 2^60 above costs is small values: the sum of a row's weights is 2^-60 (1 - 2^-8) at least, and products below
// FP32's 2^-126, 16 tokens a step, are lost beside it: 2^-70 a token.  At the other end, weights below 2^64 (BF16: 2) of
// the 2^24 tokens that a table holds leave room for values up to 2^39.
template <bool FP8>
constexpr float kAbove = FP8 ? 0.f : 60.f;

// What has become of a half's weights besides themselves: whether some are too large or not numbers (m has to move).
template <bool FP8>
struct Excess {
    uint32_t bits = 0;  // BF16: an exponent's first bit is 2 or more
    float most = 0.f;
    __device__ __forceinline__ bool any() const { return FP8 ? !(most < kMostWeight) : (bits & 0x40004000u) != 0; }
};

// 32 scores (columns 32 q ..) as weights 2^(S c - m), in pairs rounded to BF16 (half a step, 2^-8): what the matrix
// instruction takes beside BF16 values.
template <bool FP8, bool MASKED>
__device__ __forceinline__ void weigh(const HalfRow &h, int q, const uint32_t (&w)[32], float m, uint32_t *p, Excess<FP8> &ex)
{
    const float2 m2 = make_float2(-m, -m);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const int at = q * 16 + i;
        const float4 f = FP8 ? h.ks[at / 2] : make_float4(h.c, h.c, h.c, h.c);
        const float2 x =
            tc::fma2(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), make_float2(f.x, f.y), m2);
        const float2 y =
            tc::fma2(make_float2(__uint_as_float(w[2 * i + 2]), __uint_as_float(w[2 * i + 3])), make_float2(f.z, f.w), m2);
        float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y)), g = make_float2(ex2_approx(y.x), ex2_approx(y.y));
        h.drop<MASKED>(at, e, 0.f);
        h.drop<MASKED>(at + 1, g, 0.f);
        if (FP8) {
            ex.most = tc::max3(tc::max3(ex.most, e.x, e.y), g.x, g.y);
            const float4 v = h.vs[at / 2];
            e = tc::mul2(e, make_float2(v.x, v.y));
            g = tc::mul2(g, make_float2(v.z, v.w));
            h.drop<MASKED>(at, e, 0.f);  // (the scale may be anything)
            h.drop<MASKED>(at + 1, g, 0.f);
        }
        p[i] = pack_bf16x2(e.x, e.y);
        p[i + 1] = pack_bf16x2(g.x, g.y);
        if (!FP8)
            ex.bits |= p[i] | p[i + 1];
    }
}

template <bool FP8, bool MASKED>
__device__ __forceinline__ bool half_weights(const HalfRow &h, float m, uint32_t (&p)[32])
{
    Excess<FP8> ex;
    uint32_t w0[32], w1[32];
    tc::ld32(h.ts, w0);
    tc::ld32_begin(h.ts + 32, w1);
    weigh<FP8, MASKED>(h, 0, w0, m, p, ex);
    tc::loads_done(w1);
    weigh<FP8, MASKED>(h, 1, w1, m, p + 16, ex);
    return ex.any();
}

// The reference of the rows with `move` moves to the maximum of their scores, and what they have summed up so far with
// it; then the weights.  (If a wait gives up here the next one does.)
template <bool FP8, bool MASKED>
__device__ __noinline__ float move_reference(HalfRow h, bool move, float m, uint64_t *o_step, int before, volatile int *stop)
{
    const float top = top_score<FP8, MASKED>(h);
    const float mn = move ? fmaxf(top + kAbove<FP8>, m) : m;
    const float f = move ? ex2_approx(m - mn) : 1.f;
    // Once the product before this one is done, nothing else touches O.  (These scores came
    // after the product before that, so the wait is one phase behind at most.)
    if (!wait_for(o_step, (before - 1) & 1, stop))
        return m;
    tc::fence_after();
#pragma unroll 1
    for (int k = 0; k < 5; ++k) {  // (O's 64 columns and the sums' 16)
        uint32_t o[16];
        const uint32_t at = k < 4 ? h.to + k * 16 : h.tl;
        tc::ld16(at, o);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tc::st16(at, o);
    }
    uint32_t p[32];
    (void)half_weights<FP8, MASKED>(h, mn, p);
    tc::st32(h.ts, p);
    return mn;
}

// A row's first reference: of the half tile's scores.
template <bool FP8, bool MASKED>
__device__ __forceinline__ void first_reference(const HalfRow &h, float &m)
{
    if (__any_sync(kFull, m == -INFINITY)) {
        const float top = top_score<FP8, MASKED>(h);
        if (m == -INFINITY)
            m = top + kAbove<FP8>;
    }
}

// Half a key tile's scores of one query row become weights, in place (P is the first half of S's columns).  The
// reference m is taken from the row's first scores' maximum and rarely moves (see kMostWeight); -inf: nothing
// attended to so far.  The softmax's sum is of the weights as rounded, made by the matrix instruction (see make_weights).
// What is rarely taken is in functions of their own, which load the scores again: kept in registers for a second round
// over them, they cost every half their spills (2048 tokens behind 14000: 354 us where this took 266).
template <bool FP8, bool MASKED>
__device__ __forceinline__ void softmax_half(const HalfRow &h, int before, uint64_t *o_step, volatile int *stop, float &m)
{
    first_reference<FP8, MASKED>(h, m);
    uint32_t p[32];
    const bool move = half_weights<FP8, MASKED>(h, m, p);
    if (__any_sync(kFull, move))
        m = move_reference<FP8, MASKED>(h, move, m, o_step, before, stop);
    else
        tc::st32(h.ts, p);  // columns 2i, 2i + 1 of S are column i of P
    tc::wait_st();
}

// Where the partials of part i of an item lie: rows of row tile s.
__device__ __forceinline__ size_t part_rows(const Item &x, int i, int s)
{
    return ((size_t)((x.first + i) * 2 + (i == 0 ? 1 : 0)) * 2 + s) * kRowTile;
}


// Softmax warps of row tile s: thread = query row (token r / 4 of the tile, head r % 4).
template <bool FP8>
struct Softmax {
    const ChunkArgs &a;
    ChunkShared &sh;
    uint8_t *stages, *rows;  // (the warp's rows)
    int s, warp, lane, r;
    uint32_t ts, to, tq, tl;
    int loaded = 0, checks = 0, done = 0, used = 0;
    int fetched = -1, queried = -1;  // the item whose queries are in shared memory (or on their way), in tensor memory
    int met = 0;                     // times the row tile's warps have met

    __device__ __forceinline__ Softmax(const ChunkArgs &a_, ChunkShared &sh_, uint8_t *stages_, uint8_t *rows_, uint32_t tmem)
        : a(a_), sh(sh_), stages(stages_), rows(rows_ + (threadIdx.x >> 5) * 32 * kRowBytes), warp(threadIdx.x >> 5),
          lane(threadIdx.x & 31)
    {
        s = warp >> 2;
        r = (warp & 3) * 32 + lane;
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        ts = at + kColS + s * 128;
        to = at + kColO + s * 64;
        tq = at + kColQ + s * 32;
        tl = at + kColL + s * 16;
    }

    // The warps of the row tile wait for each other; false if that gave up.
    __device__ __forceinline__ bool meet()
    {
        __syncwarp();
        if (lane == 0)
            tc::mbar_arrive(&sh.group[s]);
        return wait_for(&sh.group[s], met++ & 1, &sh.stop);
    }

    // Ticket of a cut item, whose partials the row tile's threads have written: `last` for the one that
    // finishes last and has everybody's partials to read.  False if a wait gave up.
    __device__ __forceinline__ bool draw_ticket(const Item &x, bool &last)
    {
        // (what the threads have written comes before their meeting, that before the ticket, and the
        // ticket before whoever draws a later one: no fences besides)
        if (!meet())
            return false;
        if ((int)threadIdx.x == s * 128) {
            int *ticket = &a.tickets[x.first * 2 + s];
            int drawn;
            asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(drawn) : "l"(ticket) : "memory");
            sh.taken[x.me == 0][s] = 1;
            sh.last[s] = drawn == x.parts - 1;
            if (drawn == x.parts - 1)
                *ticket = 0;
        }
        if (!meet())
            return false;
        last = *(volatile int *)&sh.last[s] != 0;
        return true;
    }

    // First of the 4 rows of the warp's first token; the next token's are kTokenRow further on.
    __device__ __forceinline__ int64_t rows_at(const Item &x) const
    {
        return x.row + (s == 0 ? 0 : x.kind == plan::kPair ? plan::kRowTokens * kTokenRow : kGroup * kD) +
               (warp & 3) * 8 * kTokenRow;
    }
    // Of the warp's 8 tokens, those there are.
    __device__ __forceinline__ int live_tokens(const Item &x) const { return x.tokens(s) - (warp & 3) * 8; }

    // An item's query rows on their way to the warp's rows in shared memory: a token's four heads lie side by side.
    __device__ __forceinline__ void fetch(const Item &x)
    {
        const int live = live_tokens(x);
        const uint16_t *src = a.q + (live > 0 ? rows_at(x) + lane * 8 : 0);
        const uint32_t dst = smem_addr(rows) + lane / 8 * kRowBytes + lane % 8 * 16;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * kGroup * kRowBytes),
                         "l"(src + (i < live ? i * kTokenRow : 0)), "r"(i < live ? 16 : 0)
                         : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    // From there into tensor memory: 64 values, two to a column.  (Every product of the previous item
    // with its queries is done when its last scores are there.)
    __device__ __forceinline__ void queries()
    {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4 v = *reinterpret_cast<const uint4 *>(rows + lane * kRowBytes + i * 16);
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

    // The warp's rows in shared memory (128 bytes each) to `dst`, the next token's four `token` 16-byte chunks
    // further on and a token's `row` apart: whole lines.
    __device__ __forceinline__ void store_rows(int live, uint4 *dst, int token, int row) const
    {
        __syncwarp();
        dst += lane / 8 * row + lane % 8;
        const uint8_t *src = rows + lane / 8 * kRowBytes + lane % 8 * 16;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live)
                __stcg(dst + i * token, *reinterpret_cast<const uint4 *>(src + i * kGroup * kRowBytes));
        __syncwarp();
    }

    // Half hf of the piece's j-th key tile, whose load is in stage st.
    __device__ __forceinline__ HalfRow half_row(int st, int hf) const
    {
        HalfRow h;
        h.ts = ts + hf * kHalf;
        h.to = to;
        h.tl = tl;
        h.c = a.scale_log2;
        h.ks = reinterpret_cast<const float4 *>(sh.scales[st][0] + hf * kHalf);
        h.vs = reinterpret_cast<const float4 *>(sh.scales[st][1] + hf * kHalf);
        h.mask = make_uint2(0, 0);
        return h;
    }

    __device__ __forceinline__ void weights_there(int hf)
    {
        tc::fence_before();
        __syncwarp();
        if (lane == 0)
            tc::mbar_arrive(&sh.p_full[s][hf]);
    }

    // A masked key tile.
    __device__ __forceinline__ bool masked_tile(const Item &x, int j, int pos, float &m, int &bad, uint32_t &nan_lo,
                                                uint32_t &nan_hi)
    {
        const int seq = loaded + x.order(s, j), st = seq % kStages;
        if (FP8)  // what this thread reads of the stage itself
            if (!wait_for(&sh.full[st], (seq / kStages) & 1, &sh.stop))
                return false;
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
            HalfRow h = half_row(st, hf);
            h.mask = columns(x, x.j0 + j, hf, pos, a.window, a.sinks);
            if (!wait_for(&sh.s_full[s][hf], (done + j) & 1, &sh.stop))
                return false;
            tc::fence_after();
            softmax_half<FP8, true>(h, 2 * (done + j) + hf, &sh.o_step[s], &sh.stop, m);
            if (hf == 1) {  // (until its weights are there, the stage is this tile's)
                bad |= *(volatile int *)&sh.bad[st];
                const int check = checks + x.masked_loads(j) + (x.kind == plan::kHeads ? s : 0);
                if (!FP8 && !wait_for(&sh.checked[check % kStages], (check / kStages) & 1, &sh.stop))
                    return false;
                if (*(volatile int *)&sh.noted[st] == seq) {
                    reached(h.mask, sh.poison[st], 1, seq, nan_lo, nan_hi);
                    reached(columns(x, x.j0 + j, 0, pos, a.window, a.sinks), sh.poison[st], 0, seq, nan_lo, nan_hi);
                }
            }
            weights_there(hf);
        }
        return true;
    }

    // Key tiles j0 .. j1 - 1 of the piece, in which every row attends to every place.  The scores come 32 at a time,
    // the second on their way while the first become weights (2048 tokens behind 14000: 233 us where 64 at a
    // time took 255; the next half's first on their way as well: 282, registers that go round a loop).
    __device__ __forceinline__ bool plain_tiles(const Item &x, int j0, int j1, float &m, int &bad)
    {
#pragma unroll 1
        for (int k = 2 * j0; k < 2 * j1; ++k) {
            const int j = k >> 1, hf = k & 1, seq = loaded + x.order(s, j), st = seq % kStages;
            if (FP8 && hf == 0 && !wait_for(&sh.full[st], (seq / kStages) & 1, &sh.stop))
                return false;  // (what this thread reads of the stage itself)
            if (!wait_for(&sh.s_full[s][hf], (done + j) & 1, &sh.stop))
                return false;
            tc::fence_after();
            const HalfRow h = half_row(st, hf);
            uint32_t w0[32], w1[32], p[32];
            tc::ld32(h.ts, w0);
            if (k == 2 * j0)
                first_reference<FP8, false>(h, m);
            tc::ld32_begin(h.ts + 32, w1);
            Excess<FP8> ex;
            weigh<FP8, false>(h, 0, w0, m, p, ex);
            tc::loads_done(w1);
            weigh<FP8, false>(h, 1, w1, m, p + 16, ex);
            if (hf == 1)  // (until its weights are there, the stage is this tile's)
                bad |= *(volatile int *)&sh.bad[st];
            const bool move = ex.any();
            if (__any_sync(kFull, move))
                m = move_reference<FP8, false>(h, move, m, &sh.o_step[s], 2 * (done + j) + hf, &sh.stop);
            else
                tc::st32(h.ts, p);  // columns 2i, 2i + 1 of S are column i of P
            tc::wait_st();
            weights_there(hf);
        }
        return true;
    }

    // A piece of row tiles; false if a wait gave up.
    __device__ __forceinline__ bool tiles_piece(Feed &feed, const Item &it)
    {
        const Item x = it;
        if (queried != feed.n) {
            if (fetched != feed.n)
                fetch(x);
            queries();
            const Item *y = feed.look(1);
            if (y) {
                fetch(*y);
                fetched = feed.n + 1;
            }
        }
        const int live = live_tokens(x), nt = x.j1 - x.j0;
        const bool idle = live <= 0;  // no row of the warp is a query: it only keeps step
        const int pos = x.p0 + x.token(s) + min(r / kGroup, x.tokens(s) - 1);
        float m = -INFINITY;
        int bad = 0;
        uint32_t nan_lo = 0, nan_hi = 0;
        if (a.expire && s == 0 && used == 0) {
            *(volatile int *)&sh.stop = 1;
            return false;
        }
        for (int j = 0; j < nt;) {
            if (idle) {
                for (int hf = 0; hf < 2; ++hf) {
                    if (!wait_for(&sh.s_full[s][hf], (done + j) & 1, &sh.stop))
                        return false;
                    if (lane == 0)
                        tc::mbar_arrive(&sh.p_full[s][hf]);
                }
                ++j;
            } else if (x.masked(x.j0 + j)) {
                if (!masked_tile(x, j, pos, m, bad, nan_lo, nan_hi))
                    return false;
                ++j;
            } else {
                const int end = min(nt, (x.j0 + j < x.plain ? x.plain : x.plain1) - x.j0);
                if (!plain_tiles(x, j, end, m, bad))
                    return false;
                j = end;
            }
        }
        // the next item's first scores are made while this one's last product and its output end
        const Item *y = feed.look(1);
        if (y) {
            if (fetched != feed.n + 1)
                fetch(*y);
            queries();
            queried = feed.n + 1;
        }
        if (!wait_for(&sh.o_full[s], used & 1, &sh.stop))
            return false;
        tc::fence_after();
        float l;
        {
            uint32_t sums[16];
            tc::ld16(tl, sums);
            l = __uint_as_float(sums[0]) + (FP8 ? __uint_as_float(sums[1]) : 0.f);
        }
        if (bad && r == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
        uint32_t o[64];
        tc::ld64(to, o);
        if (nan_lo | nan_hi) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if ((i < 32 ? nan_lo : nan_hi) >> (i & 31) & 1u)
                    o[i] = 0x7fffffffu;
        }
        uint4 *own = reinterpret_cast<uint4 *>(rows + lane * kRowBytes);
        if (x.parts == 1) {
            const float f = inverse_sum(l);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = bad ? 0u : pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * f, __uint_as_float(o[8 * i + 2 * k + 1]) * f);
                own[i] = make_uint4(v[0], v[1], v[2], v[3]);
            }
            store_rows(live, reinterpret_cast<uint4 *>(a.out + rows_at(x)), kTokenRow / 8, 8);
        } else {
            const size_t at = part_rows(x, x.me, s) + (warp & 3) * 32;
#pragma unroll
            for (int q2 = 0; q2 < 2; ++q2) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    own[i] = make_uint4(o[32 * q2 + 4 * i], o[32 * q2 + 4 * i + 1], o[32 * q2 + 4 * i + 2],
                                        o[32 * q2 + 4 * i + 3]);
                store_rows(live, reinterpret_cast<uint4 *>(a.part_o + at * kD) + 8 * q2, kGroup * kD / 4, kD / 4);
            }
            if (lane / kGroup < live)
                __stcg(a.part_ml + at + lane, bad ? bad_part() : make_float2(m, l));
            bool last;
            if (!draw_ticket(x, last))
                return false;
            if (last)
                join(x, live);
        }
        if (queried == feed.n + 1) {
            const Item *z = feed.look(2);
            if (z) {
                fetch(*z);
                fetched = feed.n + 2;
            }
        }
        loaded += x.loads();
        checks += x.masked_loads(nt);
        done += nt;
        ++used;
        return true;
    }

    // The warp's rows of a cut item, of all parts: two rows at a time, 16 lanes each, 16 bytes a lane, 16 rows'
    // loads of two parts on their way at once.
    __device__ __forceinline__ void join(const Item &x, int live) const
    {
        if (live <= 0)
            return;
        const int w0 = (warp & 3) * 32, last = x.parts - 1;
        float M = -INFINITY;  // of row `lane`
        bool bad = false;
#pragma unroll 1
        for (int i = 0; i < x.parts; i += 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 ml = __ldcg(a.part_ml + part_rows(x, min(i + k, last), s) + w0 + lane);
                M = fmaxf(M, ml.x);
                bad |= is_bad_part(ml.y);
            }
        }
        const unsigned zeros = __ballot_sync(kFull, bad);
#pragma unroll 1
        for (int k0 = 0; k0 < 16; k0 += 8) {
            float l = 0.f;
            float4 o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int i = 0; i < x.parts; i += 2) {
                float2 ml[2];
                float4 v[2][8];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const size_t at = part_rows(x, min(i + n, last), s) + w0;
                    ml[n] = __ldcg(a.part_ml + at + lane);
                    const float4 *src = reinterpret_cast<const float4 *>(a.part_o + at * kD) + k0 * 32 + lane;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[n][k] = __ldcg(src + k * 32);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    // (a part without scores counts nothing; one whose scores are not numbers has no maximum either,
                    // and its sums, which are not numbers, go on.  The last part again, where there is no other, is left out.)
                    const bool none = i + n > last;
                    const float f = none ? -1.f : ml[n].x == -INFINITY ? 0.f : ex2_approx(ml[n].x - M);
                    l = none ? l : fmaf(f, ml[n].y, l);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float g = __shfl_sync(kFull, f, 2 * (k0 + k) + lane / 16);
                        if (!(g < 0.f)) {
                            o[k].x = fmaf(g, v[n][k].x, o[k].x);
                            o[k].y = fmaf(g, v[n][k].y, o[k].y);
                            o[k].z = fmaf(g, v[n][k].z, o[k].z);
                            o[k].w = fmaf(g, v[n][k].w, o[k].w);
                        }
                    }
                }
            }
            const float inv = inverse_sum(l);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int row = 2 * (k0 + k) + lane / 16;
                const float g = __shfl_sync(kFull, inv, row);
                uint2 v = make_uint2(pack_bf16x2(o[k].x * g, o[k].y * g), pack_bf16x2(o[k].z * g, o[k].w * g));
                if (zeros >> row & 1u)
                    v = make_uint2(0, 0);
                if (row / kGroup < live)
                    *reinterpret_cast<uint2 *>(a.out + rows_at(x) + row / kGroup * kTokenRow + row % kGroup * kD +
                                               lane % 16 * 4) = v;
            }
        }
    }

    __device__ __forceinline__ void run()
    {
        Feed feed(sh);
        for (const Item *x; (x = feed.look()) != nullptr; feed.let_go())
            if (!tiles_piece(feed, *x))
                break;
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
};

// ------------------------------------------------------------------ the kernel

template <bool FP8>
__global__ void __launch_bounds__(TileRun<FP8>::kThreads, 1)
chunk_kernel(const __grid_constant__ CUtensorMap tmap, const __grid_constant__ ChunkArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded address: the compiler keeps shared-memory instructions)
    uint8_t *stages = smem_raw + (-smem_addr(smem_raw) & 1023u);
    uint8_t *sums = stages + kStages * kStageSize;
    uint8_t *rows = sums + sums_size(FP8), *raws = rows + kRowsSize;
    ChunkShared &sh = *reinterpret_cast<ChunkShared *>(raws + (FP8 ? kRaws * kRawSize : 0));
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], FP8 ? kPreparers : 1);
            mbar_init(&sh.empty[i], 2);
            mbar_init(&sh.checked[i], 1);
            sh.noted[i] = -1;
        }
        for (int i = 0; i < kRaws; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], kPreparers);
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
        }
        mbar_init(&sh.group[2], kPreparers);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], TileRun<FP8>::kConsumers);
        }
        sh.stop = 0;
        sh.claimed = 0;
        sh.taken[0][0] = sh.taken[0][1] = sh.taken[1][0] = sh.taken[1][1] = 0;
        fence_barrier_init();
    }
    if (warp == kIssuer)
        tc::alloc<kCols>(&sh.tmem);
    for (int i = threadIdx.x; i < kStages * kTilePages * kPage; i += TileRun<FP8>::kThreads)
        (&sh.poison[0][0])[i].load = -1;
    if (!FP8) {
        for (int i = threadIdx.x; i < sums_size(FP8) / 4; i += TileRun<FP8>::kThreads)
            reinterpret_cast<uint32_t *>(sums)[i] = 0x3f803f80u;
        fence_proxy_async_smem();
    }
    grid_dependency_wait();
    if (a.apart && blockIdx.x == 0) {  // (see launch_singles)
        if (threadIdx.x == 0)
            asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(a.arrived), "r"(1) : "memory");
        __syncthreads();
    }
    allow_dependent_launch();
    make_plan<TileRun<FP8>>(a, sh);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sh.tmem;
    // FP8: 512 threads of 128 registers; the softmax warps take 176 and leave the others 80 (168 and 88: 2048 tokens
    // behind 63000 1366 us where this takes 1350; 184 and 72: 1452).  (Registers move by fours of warps.  BF16's
    // 384 threads have 168 each; with 512, four of its warps to go through masked tiles: 251 us for 2048 behind
    // 14000 where this takes 231.)
    if (sh.length == 0) {
        // nothing (single tokens alone): at once to the end, so that the single tokens' kernel has the SM
    } else if (warp < kLoader) {
        if constexpr (FP8)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        Softmax<FP8>(a, sh, stages, rows, tmem).run();
    } else {
        if constexpr (FP8)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == kLoader)
            loader<FP8>(&tmap, a, stages, raws, sh);
        else if (warp < kIssuer + 2)
            issuer<FP8>(stages, sums, sh, tmem, warp - kIssuer);
        else if (warp == kScheduler)
            pieces<TileRun<FP8>>(a, sh, false);
        else if (FP8)
            preparer(a, raws, stages, sums, sh);
    }
    __syncthreads();
    if (sh.stop && warp == kScheduler) {
        pieces<TileRun<FP8>>(a, sh, true);
        if ((threadIdx.x & 31) == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_TIMEOUT);
    }
    if (warp == kIssuer)
        tc::dealloc<kCols>(tmem);
}

// Workspace: the tile kernel's tickets and `arrived`, its partials, then the single tokens' own.
struct ChunkWorkspace {
    size_t tickets, ml, o;
    size_t singles() const { return tickets + ml + o; }
    size_t total() const { return singles() + single_workspace().total(); }
};

ChunkWorkspace chunk_workspace()
{
    ChunkWorkspace w;
    w.tickets = align256(((size_t)kSms * 2 + 1) * sizeof(int));
    w.ml = align256((size_t)kSms * 4 * kRowTile * sizeof(float2));
    w.o = (size_t)kSms * 4 * kRowTile * kD * sizeof(float);
    return w;
}

// Whether single tokens are a kernel's of their own: where there must be some (fewer than two tokens a sequence: 2 to
// 128 sequences of up to 600 to 16000 tokens take 0.57 to 0.89 of the time among the tiles, FP8 0.31 to 0.83), and in large
// batches.  Where there need be none, the second kernel costs what finding that out takes.  Time apart by time among the
// tiles, 1 prompt of 300 or 2 of 700 beside single tokens of up to 600, 3000 and 16000: BF16, 16 sequences 1.12 to 1.16,
// 1.15 to 1.16 and 0.96 to 0.98, 24 1.08 to 1.14, 1.09 to 1.17 and 0.93 to 0.96, 32 0.88 to 1.06, 1.02 to 1.04 and 0.91 to
// 0.93, 64 0.96 to 1.02, 0.95 to 0.96 and 0.89 to 0.91; FP8, whose tiles are dearer, 4 1.02 to 1.10, 1.07 to 1.12 and 0.94 to
// 0.97, 8 0.95 to 1.07, 0.99 to 1.04 and 0.90, 16 0.90 to 1.03, 0.89 to 0.91 and 0.76 to 0.80.
bool apart_of(bool fp8, int B, int T) { return B >= 2 && (T < 2 * B || B >= (fp8 ? 8 : 32)); }

template <bool FP8>
int launch_chunk(const pkv_pool *pool, const ChunkArgs &a, cudaStream_t s, bool pdl)
{
    const CUtensorMap *tmap = pool_tensor_map(pool);
    if (!tmap)
        return PKV_ERR_CUDA;
    constexpr int smem = 1024 + kStages * kStageSize + sums_size(FP8) + kRowsSize + (FP8 ? kRaws * kRawSize : 0) +
                         (int)sizeof(ChunkShared);
    static_assert(smem <= 227 * 1024, "shared memory of an SM");
    static PerDeviceOnce attr;
    if (const int st = ensure_smem_attr(attr, chunk_kernel<FP8>, smem); st != PKV_OK)
        return st;
    return launch_kernel(chunk_kernel<FP8>, dim3(kSms), dim3(TileRun<FP8>::kThreads), smem, s, pdl, *tmap, a);
}

}  // namespace
}  // namespace chunk
}  // namespace pkv

extern "C" size_t pkv_chunk_attention_workspace_bytes(int B, int T)
{
    return pkv::chunk::chunk_args_ok(B, T) ? pkv::chunk::chunk_workspace().total() : 0;
}

extern "C" int pkv_chunk_attention(const pkv_pool *pool, const uint16_t *q, const int32_t *bt_dev, int max_blocks,
                                   const int32_t *seq_lens_dev, const int32_t *starts_dev, int B, int T, float scale,
                                   int window, int sinks, void *workspace, size_t workspace_bytes, uint16_t *out,
                                   int32_t *dev_err_flag, void *cuda_stream, int options)
{
    using namespace pkv;
    using namespace pkv::chunk;
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
    a.arrived = a.tickets + kSms * 2;
    a.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + ws.tickets);
    a.part_o = reinterpret_cast<float *>(static_cast<char *>(workspace) + ws.tickets + ws.ml);
    a.expire = (options & PKV_STEP_TEST_EXPIRE_WAIT) ? 1 : 0;
    a.apart = false;
    a.refuses = true;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    const bool pdl = !(options & PKV_STEP_NO_PDL);
    void *singles = static_cast<char *>(workspace) + ws.singles();
    if (T == 1)
        return launch_singles(pool, a, singles, s, pdl, false);
    a.apart = apart_of(pool->kv_format == PKV_KV_FP8, B, T);
    if (const int st = pool->kv_format == PKV_KV_FP8 ? launch_chunk<true>(pool, a, s, pdl) : launch_chunk<false>(pool, a, s, pdl);
        st != PKV_OK || !a.apart)
        return st;
    return launch_singles(pool, a, singles, s, pdl, true);
}
