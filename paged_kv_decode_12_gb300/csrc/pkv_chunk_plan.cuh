// pkv_chunk_plan.cuh -- how the attention of chunks is cut into pieces of work, one run of them a CTA.
// Not part of the ABI.
//
// A sequence's new tokens make items: 64 tokens and one KV head (two row tiles of 128 query rows that go
// through the same pages); the odd last 32 tokens, or fewer, and two KV heads (a row tile each); or, in a kernel
// of their own, a sequence's single token and one KV head.  An item goes through `nt` key tiles of 128 tokens and
// costs nt * tile + item.  All items laid end to end make a line of length W, and CTA c of G works off what lies
// between c W / G and (c + 1) W / G: the work is even whatever the lengths are, and an item that crosses a border is
// cut between key tiles (not next to its ends: cut()), its parts joined by whoever finishes last.  At most one cut item begins and
// at most one goes on in a CTA, which bounds the partial results to two a CTA.
#pragma once

#include <cstdint>

#include "pkv_internal.h"

namespace pkv {
namespace plan {

constexpr int kTileTokens = 128;   // of a key tile
constexpr int kRowTokens = 32;     // of a row tile
constexpr int kLeast = 2;          // key tiles of a part

enum Kind { kEnd = 0, kPair = 1, kHeads = 2, kSingle = 3 };

// What the kinds of items cost, in a common unit.
struct Costs {
    int tile[4], item[4];
};

#define PKV_HD __host__ __device__ __forceinline__

// Places on the line are of type I: 32 bits where the line is short, because a warp by itself, one instruction behind
// the other, makes a piece of work before anything else can begin.
template <class I>
PKV_HD I imin(I a, I b) { return a < b ? a : b; }
template <class I>
PKV_HD I imax(I a, I b) { return a > b ? a : b; }

// The pages that the tokens at positions first .. last attend to: entry i is page i below `sink`, i -
// sink + from behind it.
struct PageList {
    int sink, from, count;
    PKV_HD int page(int i) const { return i < sink ? i : i - sink + from; }
    PKV_HD int tiles() const { return (count + kTileTokens / kPage - 1) / (kTileTokens / kPage); }
};

PKV_HD PageList page_list(int first, int last, int window, int sinks)
{
    PageList x;
    x.from = window && first + 1 > window ? (first + 1 - window) / kPage : 0;
    x.sink = imin((sinks + kPage - 1) / kPage, x.from);
    x.count = x.sink + last / kPage - x.from + 1;
    return x;
}

// a / b for a result below 8, as it is known to be, by comparisons.
template <class I>
PKV_HD int eighth(I a, I b)
{
    int n = 0;
    for (int i = 1; i < 8; ++i)
        n += a >= i * b;
    return n;
}

// The items of one sequence of n new tokens, the first at position c (which are below 2^24, as window and sinks are).
template <class I>
struct Sequence {
    int n, c, window, sinks;
    int pairs;       // items of 64 tokens a head; the last may be short
    bool rest;       // and one of 32 or fewer for every two heads
    int flat;        // key tiles of a pair once the window leaves the beginning (no window: beyond reach)
    int tile, item;  // costs of pairs

    PKV_HD Sequence(int n_, int c_, int window_, int sinks_, const Costs &k)
        : n(n_), c(c_), window(window_), sinks(sinks_), tile(k.tile[kPair]), item(k.item[kPair])
    {
        const int rows = (n + kRowTokens - 1) / kRowTokens;
        pairs = rows / 2;
        rest = (rows & 1) != 0;
        flat = 1 << 20;
        if (window) {
            const int lo = c + 1 - window;  // (floor of a negative number)
            const int from = lo >= 0 ? lo / kPage : -((-lo + kPage - 1) / kPage);
            const int span = (c + 2 * kRowTokens - 1) / kPage - from + 1;
            const int pages = (sinks + kPage - 1) / kPage + span;
            flat = (pages + kTileTokens / kPage - 1) / (kTileTokens / kPage);
        }
    }
    // Pages of pair r, of the rest, of a single token.
    PKV_HD PageList pair_pages(int r) const
    {
        return page_list(c + 64 * r, c + imin(64 * r + 63, n - 1), window, sinks);
    }
    PKV_HD PageList rest_pages() const { return page_list(c + 64 * pairs, c + n - 1, window, sinks); }
    PKV_HD PageList single_pages() const { return page_list(c, c, window, sinks); }

    // Cost of the first r pairs of a head, none of them the last: a pair's tiles are min((c + 63 + 64 r) /
    // 128 + 1, flat), two at a time one more each.
    PKV_HD I before(int r) const
    {
        const int a = c + 63;
        int turn = 128 * (flat - 1) - a;  // pairs below turn / 64 still grow
        turn = turn <= 0 ? 0 : (turn + 63) / 64;
        const I grow = imin(turn, r), m = grow / 2, e = grow & 1;
        const I a0 = a / 128, a1 = (a + 64) / 128;
        const I tiles = m * (a0 + a1) + m * (m - 1) + e * (a0 + m) + grow + (r - grow) * flat;
        return tiles * tile + (I)r * item;
    }
    PKV_HD I pair_cost(int r) const { return (I)pair_pages(r).tiles() * tile + item; }
    // Of all pairs of a head.
    PKV_HD I head_cost() const { return pairs ? before(pairs - 1) + pair_cost(pairs - 1) : 0; }
    PKV_HD I rest_cost(const Costs &k) const
    {
        return rest ? (I)rest_pages().tiles() * k.tile[kHeads] + k.item[kHeads] : 0;
    }
    PKV_HD I cost(const Costs &k) const { return kHkv * head_cost() + kHkv / 2 * rest_cost(k); }
    PKV_HD I single_cost(const Costs &k) const { return (I)single_pages().tiles() * k.tile[kSingle] + k.item[kSingle]; }
};

// The sequence's cost.  In 32 bits where it is below 2^29: 512 pairs a head of at most 4096 + 1 tiles at costs below 16.
PKV_HD bool short_row(int n, int tokens) { return n < 1 << 15 && tokens < 1 << 19; }
template <class I>
PKV_HD I row_cost(int n, int tokens, int window, int sinks, const Costs &k, bool single)
{
    const Sequence<I> seq(n, tokens - n, window, sinks, k);
    return single ? kHkv * seq.single_cost(k) : seq.cost(k);
}

// The line's borders: CTA c has border(c) .. border(c + 1), which are `each` or each + 1 apart.
template <class I>
struct Line {
    I length, each;
    int ctas, longer;  // CTAs, those among them, the first ones, with one more
    // The CTAs that a line is worth: parts that cost as much to begin as to do are not.
    PKV_HD Line(I length_, int most, int least) : length(length_)
    {
        ctas = (int)imax((I)1, imin(length / least, (I)most));
        each = length / ctas;
        longer = (int)(length - each * ctas);
    }
    PKV_HD I border(int c) const { return c * each + imin(c, longer); }
    // The first CTA whose end is not below x.
    PKV_HD int ending_from(I x) const
    {
        const I turn = longer * (each + 1);
        return x <= turn ? (int)((x + each) / (each + 1)) - 1 : longer + (int)((x - turn + each - 1) / each) - 1;
    }
};

// Key tiles of an item before a border that lies t into it.
template <class I>
PKV_HD int cut(I t, int nt, int tile, int item)
{
    if (t >= (I)nt * tile + item)
        return nt;
    if (t < item + (I)kLeast * tile)
        return 0;
    const int j = (int)((t - item) / tile);
    return j > nt - kLeast ? nt : j;
}

// The CTAs that take part in an item that begins at s: first .. first + count - 1.
struct Parts {
    int first, count;
};

template <class I>
PKV_HD Parts parts_of(const Line<I> &line, I s, int nt, int tile, int item)
{
    const I cost = (I)nt * tile + item;
    const I some = imin(cost, item + (I)kLeast * tile);                          // cut() > 0 from here
    const I all = imin(cost, imax(some, item + (I)(nt - kLeast + 1) * tile));    // == nt from here
    Parts p;
    p.first = line.ending_from(s + some);
    p.count = line.ending_from(s + all) - p.first + 1;
    return p;
}

}  // namespace plan
}  // namespace pkv
