// pkv_shared.cu -- decode attention for groups of sequences that share a prefix.
//
//     out[b][h] = sum_t softmax_t(scale * q[b][h] . K_t) V_t,   t < seq_lens[b],
//
// where the tokens of the first prefix_pages[i] pages are the same for every sequence of group i.
// softmax over a split axis: a part S of the tokens gives m = max, l = sum 2^(x - m) and
// o = sum 2^(x - m) V over S (x the score times log2 e); parts join by 2^(m - M), M their maximum.
//
// The prefix is one part or several (chunks).  There the n sequences of a group and the 4 query
// heads of a KV head are 4 n rows that meet the same keys: a matrix product of enough rows for the
// tensor cores (tcgen05), S = Q K^T and O += P V with Q, S, P and O in tensor memory and K and V
// in shared memory as TMA brought them.  What a sequence has behind the prefix goes through the
// grid kernel of pkv_step.cuh, beside the prefix kernel, and its units (or merge_kernel) join all.
//
// What bounds it: a page is read once a row tile pair instead of once a sequence, so bytes count
// little; 64 exponentials a row and half tile take 512 of the 1000 clocks it lasts, and the rest
// is the way from one wait to the next.  Two row tiles a CTA fill each other's gaps (256 sequences
// behind 32768 tokens: 94 us, 730 TFLOP/s).
// Tried: 16 softmax warps, with half a row each or as four sets of their own (149 us where 8 took
// 101), starting the second row tile half a step later (no change), 8 converter warps for FP8 (30.3 us
// where 4 took 30.8).
#include <cmath>

#include "pkv_step.cuh"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kTilePages = 8;                       // pages of one key tile: 128 tokens
constexpr int kHalf = kTilePages * kPage / 2;       // its halves
constexpr int kRowTile = 128;                       // query rows of one tensor-core tile
constexpr int kTileSeqs = kRowTile / kGroup;        // 32 sequences x the 4 heads of a KV head

// The groups of a call: group i is sequences starts[i] .. starts[i + 1] - 1, its prefix
// prefix_pages[i] pages in chunks of chunk_pages.
struct Groups {
    const int32_t *starts, *prefix_pages;
    int groups, max_prefix, chunk_pages, B;

    struct Group {
        int s0, n, prefix;
        bool ok;
    };
    // Group i, not ok if its bounds leave the batch or its prefix the announced range.
    __device__ __forceinline__ Group at(int i) const
    {
        Group x;
        x.s0 = starts[i];
        const int s1 = starts[i + 1];
        x.prefix = prefix_pages[i];
        x.ok = x.s0 >= 0 && s1 <= B && x.s0 < s1 && x.prefix >= 0 && x.prefix <= max_prefix;
        x.n = x.ok ? s1 - x.s0 : 0;
        return x;
    }
    __device__ __forceinline__ int chunks(int prefix) const { return (prefix + chunk_pages - 1) / chunk_pages; }
};

// The pages of a sequence behind its group's prefix; the prefix's partials come first.  MERGE:
// the units wait for the prefix's partials and merge; else merge_kernel does.
template <bool MERGE>
struct OwnPages {
    static constexpr bool kIdentity = false, kSortable = false, kLateWait = MERGE, kPublish = !MERGE, kLoops = true,
                          kFine = false;
    Groups gr;

    struct List {
        static constexpr bool kWhole = false;
        int L, prefix, slots;  // prefix < 0: the sequence is in no valid group
        __device__ __forceinline__ bool ok() const { return prefix >= 0 && (int64_t)prefix * kPage <= L; }
        __device__ __forceinline__ int count() const { return (L + kPage - 1) / kPage - prefix; }
        __device__ __forceinline__ int logical(int i) const { return i + prefix; }
        __device__ __forceinline__ int before(int j) const { return max(j - prefix, 0); }
        __device__ __forceinline__ FirstTokens tokens(int j) const { return {min(kPage, L - j * kPage)}; }
        __device__ __forceinline__ int first_slot() const { return slots; }
    };

    // (the whole warp looks for the group of b)
    __device__ __forceinline__ List list(int b, int L) const
    {
        int prefix = -1;
        for (int i = threadIdx.x & 31; i < gr.groups; i += 32) {
            const Groups::Group x = gr.at(i);
            if (x.ok && x.s0 <= b && b < x.s0 + x.n)
                prefix = x.prefix;
        }
        prefix = __reduce_max_sync(kFull, prefix);
        return {L, prefix, prefix > 0 ? gr.chunks(prefix) : 0};
    }
    __device__ __forceinline__ EmitNothing emit(int, int) const { return {}; }
    __device__ __forceinline__ void skipped(int, int, int, int) const {}
    __device__ __forceinline__ void finished(int, int, int, float, float, float *) const {}
};

// ------------------------------------------------------------------ the prefix on tensor cores

constexpr int kStageSize = kTilePages * kStageBytes;           // 32 KiB: 8 x (K rows, V rows)
constexpr int kRawSize = kTilePages * kFp8Unit;                // 17 KiB: FP8 units as they lie in the pages
constexpr int kRaws = 2;                                       // of them in flight
constexpr int kLoader = 8, kIssuer = 9, kConverter = 12;       // warps: 2 x 4 softmax, loader, two issuers, (FP8) four
constexpr int kConverters = 4;                                 // converters
constexpr int kOutRow = 32 * 4 + 16;                           // half an output row, padded to other banks
constexpr int kOutSize = 2 * kRowTile * kOutRow;               // 36 KiB: of every row
constexpr int kScales = 3 * kTilePages * kPage;                // row scales of a tile: K's, V's, 1 / V's
constexpr int kCols = 512;                                     // tensor memory, all of it
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384, kColL = 448;  // + 128 / 64 / 32 / 16 for the second tile
constexpr int kOnesSize = 16 * 128;                            // BF16 pages: 16 rows of ones, for the sums

constexpr int kStages = 4;  // (FP8: three were 12 % slower, five or a third raw unit no faster)
constexpr int prefix_threads(bool fp8) { return fp8 ? (kConverter + kConverters) * 32 : (kIssuer + 2) * 32; }

struct PrefixBars {
    uint64_t full[kStages], empty[kStages];              // a stage holds its pages / both tiles are done with it
    uint64_t raw_full[kRaws], raw_empty[kRaws];  // the same of the raw units
    uint64_t s_full[2][2], p_full[2][2];     // [row tile][half]: scores are in tensor memory / weights are
    uint64_t o_step[2];                      // one more product of weights and values is done
    uint64_t q_full[2], o_full[2];           // once an item: the queries are in / its last product is done
    uint32_t tmem;
    int stop;                                // a wait gave up
    int bad[kStages], raw_bad[kRaws];              // the tile has a bad page id
    uint64_t drained[2];
    // FP8: a stage's row scales, [K (times scale log2 e), V, 1 / V][half][64] in the order of S's columns
    float scales[kStages][kScales];
};

struct PrefixArgs {
    Groups gr;
    int num_pages;
    const uint16_t *q;   // [B][32][64]
    const int32_t *bt;
    int max_blocks;
    float scale_log2;
    float2 *part_ml;
    float *part_o;
    int max_chunks;
    int32_t *err;
    int expire;          // testing aid: the first wait for scores gives up at once (PKV_STEP_TEST_EXPIRE_WAIT)
};

// Two values, picked without an address (an indexed array would live in memory).
struct Two {
    int v0, v1;
    __device__ __forceinline__ int operator[](int s) const { return s ? v1 : v0; }
};

// A work item: two tiles of 128 query rows of one KV head, each with its run of key tiles.
struct Item {
    int g;       // KV head
    int lead;    // the sequence whose table row holds the prefix
    Two s0, ns;  // each tile's sequences (ns <= 32; 0: no such tile)
    Two chunk;   // each tile's chunk
    Two j0, np;  // its pages
    Two nt;      // its key tiles
    bool shared; // both tiles go through the same pages
    __device__ __forceinline__ int tiles(int s) const { return nt[s]; }
    // the place in the loader's order of tile s's j-th key tile: the pages of a shared run are
    // loaded once, two runs of their own alternate as long as both last (the first is no shorter)
    __device__ __forceinline__ int order(int s, int j) const { return shared ? j : j < nt.v1 ? 2 * j + s : nt.v1 + j; }
    __device__ __forceinline__ int loads() const { return shared ? nt.v0 : nt.v0 + nt.v1; }
};

// The items of the call, as a warp looks them up: lane i holds group i (of the first 32; more
// are read again for every item).  The row tiles of a group are paired and each pair goes
// through every chunk; an odd last row tile takes two chunks at a time.  Pairs that read the
// same pages are neighbours, so that the pages come from L2.
struct Items {
    const Groups &gr;
    struct Lane {
        int s0, n, prefix, chunks, items;
    } own;

    __device__ __forceinline__ explicit Items(const Groups &g) : gr(g), own(group(0)) {}

    __device__ __forceinline__ Lane group(int i0) const
    {
        const int i = i0 + (threadIdx.x & 31);
        Lane x = {0, 0, 0, 0, 0};
        if (i < gr.groups) {
            const Groups::Group gp = gr.at(i);
            const int tiles = (gp.n + kTileSeqs - 1) / kTileSeqs;
            x.s0 = gp.s0;
            x.n = gp.n;
            x.prefix = gp.prefix;
            x.chunks = gp.ok ? gr.chunks(gp.prefix) : 0;
            // (at most 8 x 2^10 pairs x 2^17 chunks)
            x.items = kHkv * (tiles / 2 * x.chunks + (tiles & 1) * ((x.chunks + 1) / 2));
        }
        return x;
    }

    // Item `it` (the whole warp); false past the last.
    __device__ __forceinline__ bool find(int it, Item &x) const
    {
        const int lane = threadIdx.x & 31;
        int local = it;
        for (int i0 = 0; i0 < gr.groups; i0 += 32) {
            const Lane gp = i0 == 0 ? own : group(i0);
            int src = 0;
            if (gr.groups > 1) {
                int end = gp.items;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(kFull, end, off);
                    if (lane >= off)
                        end += y;
                }
                const unsigned hit = __ballot_sync(kFull, local < end);
                if (!hit) {
                    local -= __shfl_sync(kFull, end, 31);
                    continue;
                }
                src = __ffs(hit) - 1;
                local -= __shfl_sync(kFull, end - gp.items, src);
            } else if (local >= __shfl_sync(kFull, gp.items, 0)) {
                return false;
            }
            const int s0 = __shfl_sync(kFull, gp.s0, src), n = __shfl_sync(kFull, gp.n, src);
            const int prefix = __shfl_sync(kFull, gp.prefix, src), nc = __shfl_sync(kFull, gp.chunks, src);
            const int nt = (n + kTileSeqs - 1) / kTileSeqs, pairs = nt / 2;
            const int paired = kHkv * pairs * nc;
            x.lead = s0;
            x.shared = local < paired;
            int r0, r1;
            if (x.shared) {
                const int q = pairs > 1 ? local / pairs : local;
                r0 = 2 * (local - q * pairs);
                r1 = r0 + 1;
                x.g = q & (kHkv - 1);
                x.chunk.v0 = x.chunk.v1 = (unsigned)q / kHkv;
            } else {
                const unsigned l = local - paired;
                r0 = r1 = nt - 1;
                x.g = l & (kHkv - 1);
                x.chunk.v0 = l / kHkv * 2;
                x.chunk.v1 = x.chunk.v0 + 1;
            }
            x.j0 = {x.chunk.v0 * gr.chunk_pages, x.chunk.v1 * gr.chunk_pages};
            x.np = {max(min(prefix - x.j0.v0, gr.chunk_pages), 0), max(min(prefix - x.j0.v1, gr.chunk_pages), 0)};
            x.nt = {(x.np.v0 + kTilePages - 1) / kTilePages, (x.np.v1 + kTilePages - 1) / kTilePages};
            x.s0 = {s0 + r0 * kTileSeqs, s0 + r1 * kTileSeqs};
            x.ns = {x.np.v0 > 0 ? min(kTileSeqs, n - r0 * kTileSeqs) : 0, x.np.v1 > 0 ? min(kTileSeqs, n - r1 * kTileSeqs) : 0};
            return true;
        }
        return false;
    }
};

// Loader: the pages of every item's key tiles into the ring of stages (FP8: of raw units).  A
// tile that the chunk does not fill repeats the chunk's last page (its weights are masked); a
// bad page id is replaced by page 0 and the tile marked.
template <bool FP8>
__device__ __forceinline__ void prefix_loader(const CUtensorMap *tmap, const PrefixArgs &a, uint8_t *ring, PrefixBars &bars)
{
    constexpr int kRing = FP8 ? kRaws : kStages, kSize = FP8 ? kRawSize : kStageSize;
    uint64_t *full = FP8 ? bars.raw_full : bars.full, *empty = FP8 ? bars.raw_empty : bars.empty;
    int *marks = FP8 ? bars.raw_bad : bars.bad;
    const int lane = threadIdx.x & 31;
    uint64_t policy;  // pages are read by several CTAs: no eviction hint
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    Item x;
    int seq = 0;
    bool go = true;
    const Items items(a.gr);
    for (int it = blockIdx.x; go && items.find(it, x); it += gridDim.x) {
        const int32_t *row = a.bt + (size_t)x.lead * a.max_blocks;
        const int most = x.tiles(0);
        int ids[2] = {0, 0};  // lane l: the id of page l of the current run of 4 key tiles
        unsigned bad[2] = {0, 0};
        for (int j = 0; j < most && go; ++j) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if ((s == 1 && x.shared) || j >= x.tiles(s) || !go)
                    continue;
                if (j % 4 == 0) {
                    ids[s] = row[x.j0[s] + min(j * kTilePages + lane, x.np[s] - 1)];
                    const bool out = ids[s] < 0 || ids[s] >= a.num_pages;
                    bad[s] = __ballot_sync(kFull, out);
                    if (out)
                        ids[s] = 0;
                }
                const int st = seq % kRing;
                if (seq >= kRing && !tc::wait_warp(&empty[st], (seq / kRing - 1) & 1, &bars.stop)) {
                    go = false;
                    continue;
                }
                const int id = __shfl_sync(kFull, ids[s], j % 4 * kTilePages + lane % kTilePages);
                if (lane == 0) {
                    marks[st] = (bad[s] >> (j % 4 * kTilePages)) & ((1u << kTilePages) - 1);
                    mbar_arrive_expect_tx(&full[st], kSize);
                }
                __syncwarp();
                if (lane < kTilePages) {
                    if (FP8)
                        fp8::tma_load_unit(ring + st * kSize + lane * kFp8Unit, tmap, &full[st], x.g, id, policy);
                    else
                        tma_load_page_head(ring + st * kSize + lane * kStageBytes, tmap, &full[st], x.g, id, policy);
                }
                ++seq;
            }
        }
    }
    if (*(volatile int *)&bars.stop)  // let the copies in flight land (bounded)
        for (int i = max(seq - kRing, 0); i < seq; ++i)
            (void)mbar_wait_warp(&full[i % kRing], (i / kRing) & 1);
}

// Two E4M3 codes as BF16 (exact: 4 significant bits, exponents in range; NaN stays NaN).
__device__ __forceinline__ uint32_t bf16x2_of_f16x2(uint32_t h)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ void bf16_of_e4m3x4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    uint32_t a, b;
    fp8::e4m3x4_to_f16x2(w, a, b);
    lo = bf16x2_of_f16x2(a);
    hi = bf16x2_of_f16x2(b);
}

// Converters (FP8; 128 threads): raw units into a stage of the BF16 layout.  The codes become
// BF16 as they are; the row scales go to the scores and the weights instead of the rows, so
// that nothing is rounded here.
__device__ __forceinline__ void prefix_converter(const PrefixArgs &a, const uint8_t *raws, uint8_t *stages, PrefixBars &bars)
{
    const int t = threadIdx.x - kConverter * 32, lane = threadIdx.x & 31;
    const Items items(a.gr);
    Item x;
    int seq = 0;
    for (int it = blockIdx.x; items.find(it, x); it += gridDim.x) {
        const int n = x.loads();
        for (int i = 0; i < n; ++i, ++seq) {
            const int rs = seq % kRaws, st = seq % kStages;
            if (!tc::wait_warp(&bars.raw_full[rs], (seq / kRaws) & 1, &bars.stop) ||
                (seq >= kStages && !tc::wait_warp(&bars.empty[st], (seq / kStages - 1) & 1, &bars.stop)))
                return;
            const uint8_t *raw = raws + rs * kRawSize;
            uint8_t *dst = stages + st * kStageSize;
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // K: 16 codes of a row, two chunks of 8 values
                const int u = t + 128 * k, page = u / 64, row = u % 64 / 4, part = u % 4;
                const uint4 c = *reinterpret_cast<const uint4 *>(raw + page * kFp8Unit + row * kD + part * 16);
                uint4 lo, hi;
                bf16_of_e4m3x4(c.x, lo.x, lo.y);
                bf16_of_e4m3x4(c.y, lo.z, lo.w);
                bf16_of_e4m3x4(c.z, hi.x, hi.y);
                bf16_of_e4m3x4(c.w, hi.z, hi.w);
                *reinterpret_cast<uint4 *>(dst + page * kStageBytes + swz(row, 2 * part)) = lo;
                *reinterpret_cast<uint4 *>(dst + page * kStageBytes + swz(row, 2 * part + 1)) = hi;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // V: 8 dims of the tokens 2 pair, 2 pair + 1, codes alternating
                const int u = t + 128 * k, page = u / 64, pair = u % 64 / 8, at = u % 8, chunk = at ^ ((2 * pair) & 7);
                const uint4 c = *reinterpret_cast<const uint4 *>(raw + page * kFp8Unit + fp8::kFp8Tile + pair * 2 * kD + at * 16);
                uint4 even, odd;
                bf16_of_e4m3x4(__byte_perm(c.x, c.y, 0x6420), even.x, even.y);
                bf16_of_e4m3x4(__byte_perm(c.z, c.w, 0x6420), even.z, even.w);
                bf16_of_e4m3x4(__byte_perm(c.x, c.y, 0x7531), odd.x, odd.y);
                bf16_of_e4m3x4(__byte_perm(c.z, c.w, 0x7531), odd.z, odd.w);
                uint8_t *v = dst + page * kStageBytes + kTileBytes;
                *reinterpret_cast<uint4 *>(v + swz(2 * pair, chunk)) = even;
                *reinterpret_cast<uint4 *>(v + swz(2 * pair + 1, chunk)) = odd;
            }
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {  // thread = (page, slot)
                const int page = t / kPage, slot = t % kPage;
                const float f = reinterpret_cast<const float *>(raw + page * kFp8Unit + kFp8UnitCodes)[kv * kPage + slot];
                float *to = bars.scales[st] + slot / 8 * 64 + page * 8 + slot % 8;
                if (kv) {  // (a scale below 2^-100, of rows of nothing, as 2^-100: weights are counted by its inverse)
                    const float v = fabsf(f) < 0x1p-100f ? 0x1p-100f : f;
                    to[128] = v;
                    to[256] = __frcp_rn(v);
                } else {
                    to[0] = f * a.scale_log2;
                }
            }
            if (t == 0)
                bars.bad[st] = bars.raw_bad[rs];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&bars.raw_empty[rs]);
                tc::mbar_arrive(&bars.full[st]);
            }
        }
    }
}

// Issuer (a converged warp, one elected thread of which issues): the matrix products of every
// item.  A key tile goes through in two halves of 64 tokens (slots 0..7 and 8..15 of its 8
// pages), each with scores of its own in tensor memory: while the softmax of one half runs, the
// other half's weights meet the values and its columns take the next tile's scores.
__device__ __forceinline__ void issue_scores(uint32_t k, uint32_t s, uint32_t q, uint64_t *done)
{
    // S[128 x 64] = Q K^T: columns 8 p + i are slot 8 h + i of page p (page stride 4 KiB)
    constexpr uint32_t kIdesc = tc::instr_desc(64, true, false), kHi = tc::smem_desc_hi(kStageBytes);
    const uint32_t lo = tc::smem_desc_lo(k, kStageBytes);
    if (tc::elect()) {
        tc::mma_ts<false>(s, q, lo, kHi, kIdesc);
#pragma unroll
        for (int i = 1; i < kD / 16; ++i)
            tc::mma_ts<true>(s, q + i * 8, lo + i * 2, kHi, kIdesc);
        tc::commit(done);
    }
    __syncwarp();
}

template <bool FIRST, bool SUM>
__device__ __forceinline__ void issue_output(uint32_t v, uint32_t o, uint32_t p, uint32_t ones, uint32_t l,
                                             uint64_t *free_stage, int uses, uint64_t *done, uint64_t *last)
{
    // O[128 x 64] += P V: 16 columns of P are 8 slots of two pages
    constexpr uint32_t kIdesc = tc::instr_desc(64, true, true), kHi = tc::smem_desc_hi(kStageBytes);
    const uint32_t lo = tc::smem_desc_lo(v, kStageBytes);
    if (tc::elect()) {
        tc::mma_ts<!FIRST>(o, p, lo, kHi, kIdesc);
#pragma unroll
        for (int i = 1; i < kHalf / 16; ++i)
            tc::mma_ts<true>(o, p + i * 8, lo + i * (2 * kStageBytes / 16), kHi, kIdesc);
        if constexpr (SUM) {  // L[128 x 16] += P 1
            constexpr uint32_t kOnes = tc::instr_desc(16, true, false), kOnesHi = tc::smem_desc_hi(1024);
            const uint32_t one = tc::smem_desc_lo(ones, 1024);
            tc::mma_ts<!FIRST>(l, p, one, kOnesHi, kOnes);
#pragma unroll
            for (int i = 1; i < kHalf / 16; ++i)
                tc::mma_ts<true>(l, p + i * 8, one, kOnesHi, kOnes);
        }
        tc::commit(done);
        if (last)
            tc::commit(last);
        if (free_stage) {
            tc::commit(free_stage);
            if (uses > 1)
                tc::commit(free_stage);
        }
    }
    __syncwarp();
}

// Each row tile has an issuer warp of its own, so that one's waits pass while the other's
// products run: the tensor cores take only a few instructions ahead.
template <bool FP8>
__device__ __forceinline__ void prefix_issuer(const PrefixArgs &a, uint8_t *stages, const uint8_t *ones, PrefixBars &bars,
                                              uint32_t tmem, int s)
{
    const uint32_t base = smem_addr(stages), one = smem_addr(ones), tl = tmem + kColL + s * 16;
    const uint32_t ts = tmem + kColS + s * 128, to = tmem + kColO + s * 64, tq = tmem + kColQ + s * 32;
    Item x;
    int loaded = 0;  // key tiles of earlier items
    int done = 0;    // of them, this row tile's
    int used = 0;    // earlier items with such a row tile
    const auto scores = [&](int j, int h) {
        const int seq = loaded + x.order(s, j), st = seq % kStages;
        if (h == 0) {
            if (!tc::wait_warp(&bars.full[st], (seq / kStages) & 1, &bars.stop))
                return false;
            tc::fence_after();
        }
        issue_scores(base + st * kStageSize + h * 1024, ts + h * kHalf, tq, &bars.s_full[s][h]);
        return true;
    };
    const auto output = [&](int j, int h, int nt) {
        if (!tc::wait_warp(&bars.p_full[s][h], (done + j) & 1, &bars.stop))
            return false;
        tc::fence_after();
        const int st = (loaded + x.order(s, j)) % kStages;
        const uint32_t v = base + st * kStageSize + kTileBytes + h * 1024, p = ts + h * kHalf;
        uint64_t *empty = h == 1 ? &bars.empty[st] : nullptr;
        uint64_t *last = h == 1 && j + 1 == nt ? &bars.o_full[s] : nullptr;
        const int uses = x.shared ? 1 : 2;  // a stage is free after two arrivals
        if (j == 0 && h == 0)
            issue_output<true, !FP8>(v, to, p, one, tl, empty, uses, &bars.o_step[s], last);
        else
            issue_output<false, !FP8>(v, to, p, one, tl, empty, uses, &bars.o_step[s], last);
        return true;
    };
    const Items items(a.gr);
    for (int it = blockIdx.x; items.find(it, x); it += gridDim.x) {
        const int nt = x.tiles(s);
        if (nt) {
            bool go = tc::wait_warp(&bars.q_full[s], used & 1, &bars.stop);
            tc::fence_after();
            go = go && scores(0, 0) && scores(0, 1);
            for (int j = 0; j < nt && go; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (go) {
                        go = output(j, h, nt);
                        if (go && j + 1 < nt)
                            go = scores(j + 1, h);
                    }
            if (!go) {  // let the products in flight end (bounded)
                if (tc::elect())
                    tc::commit(&bars.drained[s]);
                __syncwarp();
                (void)mbar_wait_warp(&bars.drained[s], 0);
                return;
            }
            ++used;
        }
        loaded += x.loads();
        done += nt;
    }
}

// What turns 64 scores into exponents and weights into the second product's operand: one
// factor, or (FP8) a factor and a scale for every column.
struct OneFactor {
    static constexpr bool kSum = false;  // the sum is made by the matrix instruction
    float c;
    __device__ __forceinline__ float2 factor(int) const { return make_float2(c, c); }
    __device__ __forceinline__ float2 weight(int, float2 e) const { return e; }
    __device__ __forceinline__ float2 counted(int, float2 e, uint32_t) const { return e; }
};

struct RowScales {
    static constexpr bool kSum = true;
    const float2 *k, *v, *inverse;  // 32 pairs of columns
    __device__ __forceinline__ float2 factor(int i) const { return k[i]; }
    __device__ __forceinline__ float2 weight(int i, float2 e) const { return tc::mul2(e, v[i]); }
    // The weight that the product holds: what was rounded, without V's scale again.
    __device__ __forceinline__ float2 counted(int i, float2, uint32_t p) const
    {
        return tc::mul2(make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u)), inverse[i]);
    }
};

// 32 scores of one query row (columns 32 k ..) as weights 2^(S c - m): their sum, and the weights
// in pairs rounded to BF16 (half a step, 2^-8) for the second product: what the matrix instruction
// takes beside BF16 values.  MASK: columns of pages from `pages` on weigh nothing.  Four chains of
// sums, so that no chain's latency is the time of the whole.
//
// BF16 pages: the softmax's sum is of the weights as rounded, made by the matrix instruction too (L
// += P 1, 16 equal columns), so that the quotient has none of their rounding where few weights make
// it.  256 sequences behind 32768 tokens: error 0.0017 in 94 us, where the sum of the unrounded
// weights, which this function returns, gives 0.0023 in 92, and unpacking the rounded ones took 108.
// FP8 pages: what is rounded is the weight times V's row scale; the sum takes it times the scale's
// inverse (error 0.0017 instead of 0.0023; 72 sequences in 5 groups 32 us instead of 31).
template <bool MASK, class Scale>
__device__ __forceinline__ float make_weights(uint32_t ts, int k, const Scale &sc, int pages, float m, uint32_t (&pk)[16])
{
    uint32_t w[32];
    tc::ld32(ts + k * 32, w);
    float2 sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sum[i] = make_float2(0.f, 0.f);
    const float2 m2 = make_float2(-m, -m);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 x =
            tc::fma2(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), sc.factor(k * 16 + i), m2);
        float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        if (MASK && !(k * 4 + i / 4 < pages))
            e = make_float2(0.f, 0.f);
        const float2 p = sc.weight(k * 16 + i, e);
        pk[i] = pack_bf16x2(p.x, p.y);
        sum[i % 4] = tc::add2(sum[i % 4], sc.counted(k * 16 + i, e, pk[i]));
    }
    const float2 s = tc::add2(tc::add2(sum[0], sum[1]), tc::add2(sum[2], sum[3]));
    return s.x + s.y;
}

// Their maximum, times the factors.
template <bool MASK, class Scale>
__device__ __forceinline__ float max_score(uint32_t ts, int k, const Scale &sc, int pages)
{
    uint32_t w[32];
    tc::ld32(ts + k * 32, w);
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 x = tc::mul2(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), sc.factor(k * 16 + i));
        if (!MASK || k * 4 + i / 4 < pages)
            mx = tc::max3(mx, x.x, x.y);
    }
    return mx;
}

// The reference m of a row's softmax is its first half tile's maximum, and it stays until a
// half tile's weights sum to 2^64 or more: FP32 and BF16 hold 2^127, so m, l and O remain a
// valid log-sum-exp triple that far above m, and no maximum is taken on the way.  (Moving m for
// every score 2^8 above it, as narrower types need, made most half tiles of 32 rows rescale O.)
// O is finite for values up to 2^45: 2^64 times that, over at most 2^18 half tiles.
constexpr float kMostWeight = 18446744073709551616.f;

// An item's first half tile: the row's maximum.  (Not inlined: the loop would pay for its
// registers; 256 sequences behind 32768 tokens 94.5 us instead of 95.1, though 4 behind 512 tokens
// 7.5 instead of 7.2.)
template <class Scale>
__device__ __noinline__ float first_reference(uint32_t ts, Scale sc, int pages)
{
    return fmaxf(max_score<true>(ts, 0, sc, pages), max_score<true>(ts, 1, sc, pages));
}

// Half a key tile's scores of one query row become weights, in place: P is the first half of
// S's columns.  MASK: only the first `pages` pages of the tile count.  Returns false if a wait
// gave up.
template <bool MASK, class Scale>
__device__ __forceinline__ bool softmax_half(uint32_t ts, uint32_t to, uint32_t tl, const Scale &sc, int pages, int before,
                                             uint64_t *o_step, volatile int *stop, float &m, float &l)
{
    uint32_t p0[16], p1[16];
    float s = make_weights<MASK>(ts, 0, sc, pages, m, p0) + make_weights<MASK>(ts, 1, sc, pages, m, p1);
    const bool move = !(s < kMostWeight);
    if (__any_sync(kFull, move)) {
        const float top = fmaxf(max_score<MASK>(ts, 0, sc, pages), max_score<MASK>(ts, 1, sc, pages));
        const float mn = move ? fmaxf(top, m) : m;
        const float f = ex2_approx(m - mn);  // 1 where the reference stays
        m = mn;
        l *= f;
        s = make_weights<MASK>(ts, 0, sc, pages, m, p0) + make_weights<MASK>(ts, 1, sc, pages, m, p1);
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

// Softmax warps of row tile s: thread = query row (sequence r / 4 of the tile, head r % 4).
template <bool FP8>
__device__ __forceinline__ void prefix_softmax(const PrefixArgs &a, PrefixBars &bars, uint32_t tmem, int s, uint8_t *out)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + kColS + s * 128, to = tmem + lanes + kColO + s * 64,
                   tq = tmem + lanes + kColQ + s * 32, tl = tmem + lanes + kColL + s * 16;
    const Items items(a.gr);
    int it = blockIdx.x;
    int loaded = 0, done = 0, used = 0;
    // The next item with such a row tile, from item `it` on; `skipped` counts the key tiles of
    // those without.
    const auto next = [&](Item &x, int &skipped) {
        skipped = 0;
        for (; items.find(it, x); it += gridDim.x) {
            if (x.tiles(s))
                return true;
            skipped += x.loads();
        }
        return false;
    };
    // An item's query rows into tensor memory: 64 values, two to a column.  (Every product of the
    // previous item with its queries is done when its last scores are there.)
    const auto queries = [&](const Item &x) {
        const bool live = r / kGroup < x.ns[s];
        const int b = x.s0[s] + r / kGroup, h = x.g * kGroup + r % kGroup;
        uint32_t w[32];
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ((size_t)b * kHq + h) * kD);
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
            tc::mbar_arrive(&bars.q_full[s]);
    };
    Item x, y;
    int skipped;
    bool more = next(x, skipped);
    if (more)
        queries(x);
    while (more) {
        loaded += skipped;
        const int nt = x.tiles(s);
        const bool idle = (warp & 3) * 32 >= x.ns[s] * kGroup;  // no row of the warp is a query: it only keeps step
        float m = 0.f, l = 0.f;
        int bad = 0;
        for (int j = 0; j < nt; ++j) {
            const int pages = x.np[s] - j * kTilePages;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                if (a.expire && s == 0 && used == 0 && blockIdx.x == 0) {
                    *(volatile int *)&bars.stop = 1;
                    return;
                }
                if (!tc::wait_warp(&bars.s_full[s][hf], (done + j) & 1, &bars.stop))
                    return;
                if (idle) {
                    if (lane == 0)
                        tc::mbar_arrive(&bars.p_full[s][hf]);
                    continue;
                }
                tc::fence_after();
                const int before = 2 * (done + j) + hf;  // products of this row tile so far
                const int seq = loaded + x.order(s, j), st = seq % kStages;
                const auto half = [&](const auto &sc) {
                    if (j == 0 && hf == 0)
                        m = first_reference(ts, sc, pages);
                    return pages >= kTilePages
                               ? softmax_half<false>(ts + hf * kHalf, to, tl, sc, kTilePages, before, &bars.o_step[s], &bars.stop,
                                                     m, l)
                               : softmax_half<true>(ts + hf * kHalf, to, tl, sc, pages, before, &bars.o_step[s], &bars.stop, m,
                                                    l);
                };
                bool go;
                if constexpr (FP8) {
                    // the scales are the converters' writes (the stage is full long since)
                    if (hf == 0 && !tc::wait_warp(&bars.full[st], (seq / kStages) & 1, &bars.stop))
                        return;
                    const float2 *sc = reinterpret_cast<const float2 *>(bars.scales[st]) + hf * 32;
                    go = half(RowScales{sc, sc + 64, sc + 128});
                } else {
                    go = half(OneFactor{a.scale_log2});
                }
                if (!go)
                    return;
                if (hf == 0)
                    bad |= *(volatile int *)&bars.bad[st];
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(&bars.p_full[s][hf]);
            }
        }
        // the next item's first scores are made while this one's last product and its output end
        it += gridDim.x;
        more = next(y, skipped);
        if (more)
            queries(y);
        if (!tc::wait_warp(&bars.o_full[s], used & 1, &bars.stop))
            return;
        tc::fence_after();
        // The chunk's partial; with a bad page id it is empty.  A thread's row goes through shared
        // memory, so that the warp writes whole lines: 128 bytes of four rows at once.
        if constexpr (!FP8) {
            uint32_t sums[16];
            tc::ld16(tl, sums);
            l = __uint_as_float(sums[0]);
        }
        const int ns = x.ns[s] - (warp & 3) * 8;  // of the warp's 8 sequences, those there are
        const size_t first = ((size_t)(x.s0[s] + (warp & 3) * 8) * kHq + x.g * kGroup) * a.max_chunks + x.chunk[s];
        const size_t per_seq = (size_t)kHq * a.max_chunks;
        float4 *own = reinterpret_cast<float4 *>(out + lane * kOutRow);
        float4 *dst = reinterpret_cast<float4 *>(a.part_o + (first + (size_t)(lane / 8) * a.max_chunks) * kD) + lane % 8;
        const float4 *line = reinterpret_cast<const float4 *>(out + lane / 8 * kOutRow) + lane % 8;
#pragma unroll
        for (int q2 = 0; q2 < 2; ++q2) {
            uint32_t w[32];
            tc::ld32(to + q2 * 32, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                own[i] = bad ? make_float4(0.f, 0.f, 0.f, 0.f)
                             : make_float4(__uint_as_float(w[4 * i]), __uint_as_float(w[4 * i + 1]),
                                           __uint_as_float(w[4 * i + 2]), __uint_as_float(w[4 * i + 3]));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i)  // sequence i, head lane / 8
                if (i < ns)
                    dst[i * per_seq * (kD / 4) + q2 * 8] = line[i * 4 * (kOutRow / 16)];
            __syncwarp();
        }
        if (lane / kGroup < ns)
            a.part_ml[first + lane / kGroup * per_seq + (size_t)(lane % kGroup) * a.max_chunks] =
                bad ? make_float2(-INFINITY, 0.f) : make_float2(m, l);
        if (bad && r == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
        loaded += x.loads();
        done += nt;
        ++used;
        x = y;
    }
}

template <bool FP8>
__global__ void __launch_bounds__(prefix_threads(FP8), 1)
prefix_kernel(const __grid_constant__ CUtensorMap tmap, PrefixArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded address: the compiler keeps shared-memory instructions)
    uint8_t *stages = smem_raw + (-smem_addr(smem_raw) & 1023u);
    uint8_t *outs = stages + kStages * kStageSize;
    uint8_t *raws = outs + kOutSize;  // (BF16 pages: the ones)
    PrefixBars &bars = *reinterpret_cast<PrefixBars *>(raws + (FP8 ? kRaws * kRawSize : kOnesSize));
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars.full[i], FP8 ? kConverters : 1);
            mbar_init(&bars.empty[i], 2);
        }
        for (int i = 0; i < kRaws; ++i) {
            mbar_init(&bars.raw_full[i], 1);
            mbar_init(&bars.raw_empty[i], kConverters);
        }
        for (int s = 0; s < 2; ++s) {
            for (int h = 0; h < 2; ++h) {
                mbar_init(&bars.s_full[s][h], 1);
                mbar_init(&bars.p_full[s][h], 4);
            }
            mbar_init(&bars.q_full[s], 4);
            mbar_init(&bars.o_step[s], 1);
            mbar_init(&bars.o_full[s], 1);
            mbar_init(&bars.drained[s], 1);
        }
        bars.stop = 0;
        fence_barrier_init();
    }
    if (warp == kIssuer)
        tc::alloc<kCols>(&bars.tmem);
    if (!FP8) {
        for (int i = threadIdx.x; i < kOnesSize / 4; i += prefix_threads(FP8))
            reinterpret_cast<uint32_t *>(raws)[i] = 0x3f803f80u;
        fence_proxy_async_smem();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = bars.tmem;
    grid_dependency_wait();
    allow_dependent_launch();  // the sequences' own pages need nothing of this kernel until they merge
    // FP8: 512 threads of 128 registers; the softmax warps take 168, so that none spill, and leave the
    // others 88.  (Registers move by fours of warps: warp 11 only fills up its four.)
    if (warp < kLoader) {
        if constexpr (FP8)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        prefix_softmax<FP8>(a, bars, tmem, warp >> 2, outs + warp * (32 * kOutRow));
    } else {
        if constexpr (FP8)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == kLoader)
            prefix_loader<FP8>(&tmap, a, FP8 ? raws : stages, bars);
        else if (FP8 && warp >= kConverter)
            prefix_converter(a, raws, stages, bars);
        else if (warp < kIssuer + 2)
            prefix_issuer<FP8>(a, stages, raws, bars, tmem, warp - kIssuer);
    }
    __syncthreads();
    if (threadIdx.x == 0 && bars.stop && a.err)
        atomicOr(a.err, PKV_DEVERR_TIMEOUT);
    if (warp == kIssuer)
        tc::dealloc<kCols>(tmem);
}

constexpr int kSms = 152;

// Pages per prefix chunk where the caller leaves it to the library: the chunk count whose waves
// of work items (two row tiles each, one CTA per SM) take the least time, in key tiles (BF16 pages
// 1.05 us, FP8 pages, which are converted, 1.85 us): an item costs 3.3 (1) besides its own, and
// every chunk 0.42 (0.12) of merging and 0.5 (0.1) more for every 256 sequences.  Of several
// groups the others are taken to be half as long as the longest.  Measured with chunks of 8 / 16 /
// 32 / 64 / 128 / 512 pages (us): 256 sequences, 2048 pages 323 / 216 / 151 / 115 / 101 / 93; 64
// sequences, 128 pages 21 / 19 / 16 / 19 / 28; 16 sequences, 512 pages 24 / 16 / 14 / 17 / 25 / 64, FP8
// 27 / 20 / 20 / 27 / 43 / 102; 200 sequences in 3 groups, 500 FP8 pages 69 / 53 / 45 / 41 / 52; 4
// sequences, 32 pages 7.6 / 8.7 / 9.8.
int default_prefix_chunk(int B, int groups, int max_prefix, bool fp8)
{
    const int tiles = (max_prefix + kTilePages - 1) / kTilePages;
    const double row_tiles = (B + kTileSeqs - 1) / kTileSeqs + (groups - 1) / 2.0;
    const double item = fp8 ? 1.0 : 3.3, chunk = fp8 ? 0.12 + 0.1 * B / 256 : 0.42 + 0.5 * B / 256;
    int best = tiles;
    double best_cost = 1e30;
    for (int chunks = 1; chunks <= tiles && chunks <= 64; ++chunks) {
        const int per = (tiles + chunks - 1) / chunks;
        const double items = kHkv * row_tiles * ((tiles + per - 1) / per) / 2;
        const double cost = std::ceil(items / kSms) * (per + item) + chunk * chunks;
        if (cost < best_cost) {
            best_cost = cost;
            best = per;
        }
    }
    return best * kTilePages;
}

// What a call's host-side arguments settle.
struct SharedPlan {
    int own_ppc, prefix_chunk, prefix_slots, max_chunks;
    int64_t max_items;
    bool merge_apart;
};

SharedPlan shared_plan(int B, int max_blocks, int groups, int max_prefix, int ppc, int prefix_ppc, bool fp8)
{
    SharedPlan p;
    // (32 pages at most: the width of the table says little about what is behind the prefixes)
    p.own_ppc = ppc ? ppc : std::min(default_chunk(B, max_blocks, 2), 32);
    p.prefix_chunk = kTilePages;
    p.prefix_slots = 0;
    p.max_items = 0;
    if (max_prefix > 0) {
        const int whole = (max_prefix + kTilePages - 1) / kTilePages * kTilePages;
        p.prefix_chunk = prefix_ppc ? (int)std::min<int64_t>(whole, ((int64_t)prefix_ppc + kTilePages - 1) / kTilePages * kTilePages)
                                    : default_prefix_chunk(B, groups, max_prefix, fp8);
        p.prefix_slots = (max_prefix + p.prefix_chunk - 1) / p.prefix_chunk;
        // sum over groups of ceil(n / 64) row-tile pairs, each in every chunk
        p.max_items = (int64_t)kHkv * ((B + (int64_t)(2 * kTileSeqs - 1) * groups) / (2 * kTileSeqs)) * p.prefix_slots;
    }
    p.max_chunks = p.prefix_slots + (max_blocks + p.own_ppc - 1) / p.own_ppc;
    p.merge_apart = p.max_items > 0 && B * kHkv > kSms;
    return p;
}

template <bool FP8>
int launch_prefix(const pkv_pool *pool, const PrefixArgs &a, int64_t max_items, cudaStream_t s, bool pdl)
{
    const CUtensorMap *tmap = pool_tensor_map(pool);
    if (!tmap)
        return PKV_ERR_CUDA;
    constexpr int smem =
        1024 + kStages * kStageSize + kOutSize + (FP8 ? kRaws * kRawSize : kOnesSize) + (int)sizeof(PrefixBars);
    static PerDeviceOnce attr;
    if (const int st = ensure_smem_attr(attr, prefix_kernel<FP8>, smem); st != PKV_OK)
        return st;
    const dim3 grid((unsigned)std::min<int64_t>(max_items, kSms));
    return launch_kernel(prefix_kernel<FP8>, grid, dim3(prefix_threads(FP8)), smem, s, pdl, *tmap, a);
}

// The partials of one (sequence, KV head): the prefix's chunks, then its own.
__global__ void __launch_bounds__(kThreads) merge_kernel(StepArgs a, Groups gr)
{
    const int g = blockIdx.x, b = blockIdx.y;
    const int L = a.seq_lens[b];
    const auto list = OwnPages<false>{gr}.list(b, L);
    grid_dependency_wait();
    allow_dependent_launch();
    if (!length_ok(a, L) || !list.ok())
        return;  // zeros, written by the units' kernel
    const int n = list.first_slot() + max(1, (list.count() + a.pages_per_chunk - 1) / a.pages_per_chunk);
    const int h = g * kGroup + (threadIdx.x >> 5), dp = threadIdx.x & 31;
    const size_t base = ((size_t)b * kHq + h) * a.max_chunks;
    float ls, r0, r1;
    merge_eights(a.part_ml + base, reinterpret_cast<const float2 *>(a.part_o + base * kD) + dp, n, ls, r0, r1);
    reinterpret_cast<uint32_t *>(a.out + ((size_t)b * kHq + h) * kD)[dp] = finish_pair(r0, r1, ls);
}

bool shared_args_ok(int B, int max_blocks, int groups, int max_prefix_pages, int pages_per_chunk,
                    int prefix_pages_per_chunk)
{
    return B >= 1 && B <= 65535 && max_blocks >= 1 && max_blocks <= (1 << 20) && groups >= 1 && groups <= B &&
           max_prefix_pages >= 0 && max_prefix_pages <= max_blocks && pages_per_chunk >= 0 &&
           pages_per_chunk <= kMaxPagesPerChunk && prefix_pages_per_chunk >= 0;
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_decode_shared_workspace_bytes(int B, int max_blocks, int groups, int max_prefix_pages,
                                                    int pages_per_chunk, int prefix_pages_per_chunk)
{
    using namespace pkv;
    if (!shared_args_ok(B, max_blocks, groups, max_prefix_pages, pages_per_chunk, prefix_pages_per_chunk))
        return 0;
    // (for either page format: the library's chunks differ)
    size_t most = 0;
    for (const bool fp8 : {false, true})
        most = std::max(most, workspace_layout(B, shared_plan(B, max_blocks, groups, max_prefix_pages, pages_per_chunk,
                                                              prefix_pages_per_chunk, fp8)
                                                      .max_chunks)
                                  .total());
    return most;
}

extern "C" int pkv_decode_shared(const pkv_pool *pool, const uint16_t *q, const int32_t *bt_dev, int max_blocks,
                                 const int32_t *seq_lens_dev, int B, const int32_t *group_starts_dev,
                                 const int32_t *prefix_pages_dev, int groups, int max_prefix_pages, float scale,
                                 int pages_per_chunk, int prefix_pages_per_chunk, void *workspace,
                                 size_t workspace_bytes, uint16_t *out, int32_t *dev_err_flag, void *cuda_stream,
                                 int options)
{
    using namespace pkv;
    if (!pool || !q || !bt_dev || !seq_lens_dev || !group_starts_dev || !prefix_pages_dev || !workspace || !out ||
        !shared_args_ok(B, max_blocks, groups, max_prefix_pages, pages_per_chunk, prefix_pages_per_chunk))
        return PKV_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < INFINITY))
        return PKV_ERR_INVALID_ARG;
    const uintptr_t align =
        reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(workspace);
    if (align & 15u)
        return PKV_ERR_INVALID_ARG;
    if (workspace_bytes < pkv_decode_shared_workspace_bytes(B, max_blocks, groups, max_prefix_pages, pages_per_chunk,
                                                            prefix_pages_per_chunk))
        return PKV_ERR_WORKSPACE_TOO_SMALL;
    const SharedPlan plan =
        shared_plan(B, max_blocks, groups, max_prefix_pages, pages_per_chunk, prefix_pages_per_chunk,
                    pool->kv_format == PKV_KV_FP8);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    const Groups gr = {group_starts_dev, prefix_pages_dev, groups, max_prefix_pages, plan.prefix_chunk, B};
    StepArgs a = {};
    a.q = const_cast<uint16_t *>(q);
    a.bt = bt_dev;
    a.seq_lens = seq_lens_dev;
    a.max_pos = INT_MAX;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.err = dev_err_flag;
    if (plan.max_items > INT32_MAX)
        return PKV_ERR_INVALID_ARG;
    // both launches check the options; the first is the one that must not run if they are refused
    if (const int st = check_options<OwnPages<true>>(pool, B, max_blocks, plan.own_ppc, options); st != PKV_OK)
        return st;
    const bool pdl = take_pdl_permission(pool, s, !(options & PKV_STEP_NO_PDL));
    if (plan.max_items > 0) {
        const WorkspaceLayout ws = workspace_layout(B, plan.max_chunks);
        PrefixArgs p;
        p.gr = gr;
        p.num_pages = pool->num_pages;
        p.q = q;
        p.bt = bt_dev;
        p.max_blocks = max_blocks;
        p.scale_log2 = a.scale_log2;
        p.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + ws.ml_offset());
        p.part_o = reinterpret_cast<float *>(static_cast<char *>(workspace) + ws.o_offset());
        p.max_chunks = plan.max_chunks;
        p.err = dev_err_flag;
        p.expire = (options & PKV_STEP_TEST_EXPIRE_WAIT) ? 1 : 0;
        if (const int st = pool->kv_format == PKV_KV_FP8 ? launch_prefix<true>(pool, p, plan.max_items, s, pdl)
                                                         : launch_prefix<false>(pool, p, plan.max_items, s, pdl);
            st != PKV_OK)
            return st;
    }
    // The second launch begins beside the first.  A few units wait for it and merge; many would
    // keep each other from starting, so they only publish, and a third launch merges.
    // (With no first launch the second waits for what came before the call.)
    const int first = plan.max_items > 0 ? options : options | PKV_STEP_NO_PDL;
    if (!plan.merge_apart)
        return launch_fused<false>(pool, a, OwnPages<true>{gr}, B, max_blocks, max_blocks, plan.prefix_slots, plan.own_ppc,
                                   workspace, s, first, true);
    if (const int st = launch_fused<false>(pool, a, OwnPages<false>{gr}, B, max_blocks, max_blocks, plan.prefix_slots,
                                           plan.own_ppc, workspace, s, first, true);
        st != PKV_OK)
        return st;
    return launch_kernel(merge_kernel, dim3(kHkv, B), dim3(kThreads), 0, s, !(options & PKV_STEP_NO_PDL), a, gr);
}
