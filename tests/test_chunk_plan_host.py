"""CPU checks of how the attention of chunks shares its work out (pkv_chunk_plan.cuh is host code as well): costs in 32
and in 64 bits, the pages of every item, and the pieces that the CTAs make of a line."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")

SOURCE = """
#include "pkv_chunk_plan.cuh"
using namespace pkv::plan;

// [0] total cost of a sequence, then of every item in the line's order: cost, tiles, kind, first page, pages
template <class I>
static int64_t items(int n, int c, int window, int sinks, const Costs &k, bool single, int64_t *out, int most)
{
    const Sequence<I> s(n, c, window, sinks, k);
    int64_t count = 0;
    const auto put = [&](int64_t cost, const PageList &p, int kind) {
        if (count < most) {
            const int64_t row[6] = {cost, p.tiles(), kind, p.sink, p.from, p.count};
            for (int i = 0; i < 6; ++i)
                out[count * 6 + i] = row[i];
        }
        ++count;
    };
    if (single) {
        for (int g = 0; g < pkv::kHkv; ++g)
            put(s.single_cost(k), s.single_pages(), kSingle);
        return count;
    }
    for (int g = 0; g < pkv::kHkv; ++g)
        for (int r = 0; r < s.pairs; ++r)  // (a pair's place is the cost of those before it)
            put((r + 1 < s.pairs ? s.before(r + 1) : s.head_cost()) - s.before(r), s.pair_pages(r), kPair);
    for (int h = 0; s.rest && h < pkv::kHkv / 2; ++h)
        put(s.rest_cost(k), s.rest_pages(), kHeads);
    return count;
}

template <class I>
static int pieces(int64_t length, int most, int least, int64_t n, const int64_t *rows, const int *tile, const int *item, int *out)
{
    const Line<I> line((I)length, most, least);
    if (line.border(line.ctas) != line.length)
        return -1;
    int64_t at = 0;
    int cta = 0;
    for (int64_t i = 0; i < n; ++i) {
        const int64_t cost = rows[i * 6], nt = rows[i * 6 + 1], kind = rows[i * 6 + 2];
        while (cta > 0 && line.border(cta) > at)
            --cta;
        while (line.border(cta + 1) <= at)
            ++cta;
        const Parts p = parts_of<I>(line, (I)at, (int)nt, tile[kind], item[kind]);
        int done = 0, parts = 0, first = -1;
        for (int c = cta; c < line.ctas && line.border(c) < at + cost; ++c) {  // (all CTAs that meet the item)
            const int j0 = line.border(c) <= at ? 0 : cut<I>((I)(line.border(c) - at), (int)nt, tile[kind], item[kind]);
            const int j1 = cut<I>((I)(line.border(c + 1) - at), (int)nt, tile[kind], item[kind]);
            if (j0 >= j1)
                continue;
            if (j0 != done || (first >= 0 && c != first + parts))
                return -2;  // a gap, or a CTA left out
            done = j1;
            first = first < 0 ? c : first;
            // of cut items one begins and one goes on in a CTA at most
            if ((j0 > 0 || j1 < nt) && ++out[c * 2 + (j0 == 0)] > 1)
                return -3;
            ++parts;
        }
        if (done != nt || first != p.first || parts != p.count)
            return -4;
        at += cost;
    }
    return at == length ? line.ctas : -5;
}

extern "C" {
int64_t plan_items(int wide, int n, int c, int window, int sinks, const int *tile, const int *item, int single, int64_t *out, int most)
{
    Costs k;
    for (int i = 0; i < 4; ++i) {
        k.tile[i] = tile[i];
        k.item[i] = item[i];
    }
    return wide ? items<int64_t>(n, c, window, sinks, k, single != 0, out, most) : items<int>(n, c, window, sinks, k, single != 0, out, most);
}
int64_t plan_cost(int wide, int n, int tokens, int window, int sinks, const int *tile, const int *item, int single)
{
    Costs k;
    for (int i = 0; i < 4; ++i) {
        k.tile[i] = tile[i];
        k.item[i] = item[i];
    }
    return wide ? row_cost<int64_t>(n, tokens, window, sinks, k, single != 0) : row_cost<int>(n, tokens, window, sinks, k, single != 0);
}
int plan_short(int n, int tokens) { return short_row(n, tokens); }
int plan_pieces(int wide, int64_t length, int most, int least, int64_t n, const int64_t *rows, const int *tile, const int *item, int *out)
{
    return wide ? pieces<int64_t>(length, most, least, n, rows, tile, item, out) : pieces<int>(length, most, least, n, rows, tile, item, out);
}
}
"""

# (tile, item) costs of the kinds none, pair, two heads, single and the least run of a CTA, as the kernels have them
KERNELS = {"bf16": ((0, 8, 9, 0), (0, 24, 24, 0), 32), "fp8": ((0, 14, 16, 0), (0, 38, 38, 0), 32),
           "single bf16": ((0, 0, 0, 6), (0, 0, 0, 8), 20), "single fp8": ((0, 0, 0, 4), (0, 0, 0, 8), 20)}


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", f"{CUDA}/include", "-I",
                    os.path.join(ROOT, "paged_kv_decode_12_gb300", "csrc"), "-o", str(d / "plan.so"), str(d / "plan.cpp")],
                   check=True)
    return Plan(ctypes.CDLL(str(d / "plan.so")))


class Plan:
    def __init__(self, L):
        self.L = L
        L.plan_items.restype = L.plan_cost.restype = ctypes.c_int64

    @staticmethod
    def ints(x):
        return (ctypes.c_int * 4)(*x)

    def items(self, wide, n, c, window, sinks, kernel):
        tile, item, _ = KERNELS[kernel]
        most = 8 * (n // 64 + 2)
        out = np.zeros((most, 6), np.int64)
        count = self.L.plan_items(wide, n, c, window, sinks, self.ints(tile), self.ints(item), kernel.startswith("single"),
                                  out.ctypes.data_as(ctypes.c_void_p), most)
        assert count <= most
        return out[:count]

    def cost(self, wide, n, tokens, window, sinks, kernel):
        tile, item, _ = KERNELS[kernel]
        return self.L.plan_cost(wide, n, tokens, window, sinks, self.ints(tile), self.ints(item), kernel.startswith("single"))

    def pieces(self, wide, rows, kernel, ctas=152):
        tile, item, least = KERNELS[kernel]
        rows = np.ascontiguousarray(rows)
        seen = np.zeros(2 * ctas + 2, np.int32)
        return self.L.plan_pieces(wide, ctypes.c_int64(int(rows[:, 0].sum())), ctas, least, ctypes.c_int64(len(rows)),
                                  rows.ctypes.data_as(ctypes.c_void_p), self.ints(tile), self.ints(item),
                                  seen.ctypes.data_as(ctypes.c_void_p))


def pages_of(first, last, window, sinks):
    """Pages that hold a token which one of the tokens at positions first .. last attends to."""
    p = np.arange(first, last + 1)
    if not window:
        return np.arange(last // 16 + 1)
    lo = np.maximum(p + 1 - window, 0)
    pages = set(range(int(lo.min()) // 16, last // 16 + 1))
    pages |= set(range(0, -(-min(sinks, int(lo.max())) // 16)))
    return np.array(sorted(pages))


def check_items(rows, n, c, window, sinks, kernel):
    tile, item, _ = KERNELS[kernel]
    pairs = (-(-n // 32)) // 2
    for i, (cost, nt, kind, sink, start, count) in enumerate(rows.tolist()):
        first = c + (64 * (i % pairs) if kind == 1 else 64 * pairs if kind == 2 else 0)
        last = min(first + (63 if kind == 1 else 31 if kind == 2 else 0), c + n - 1)
        have = np.concatenate([np.arange(sink), start + np.arange(count - sink)])
        need = pages_of(first, last, window, sinks)
        assert np.isin(need, have).all() and np.unique(have).size == have.size and have[-1] == last // 16
        assert have.size <= need.size + 1                          # (a window's sinks may end in a page of it)
        assert nt == -(-count // 8) and cost == nt * tile[kind] + item[kind]


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_items_of_random_sequences(plan, kernel):
    r = np.random.default_rng(1)
    for _ in range(400):
        n = 1 if kernel.startswith("single") else int(np.exp(r.uniform(0, np.log(700))))
        c = int(np.exp(r.uniform(0, np.log(9000)))) * int(r.integers(0, 2))
        window = int(np.exp(r.uniform(0, np.log(5000)))) * int(r.integers(0, 2))
        sinks = int(r.integers(0, 120)) if window else 0
        rows = plan.items(1, n, c, window, sinks, kernel)
        assert np.array_equal(rows, plan.items(0, n, c, window, sinks, kernel))
        total = int(rows[:, 0].sum())
        assert total == plan.cost(1, n, c + n, window, sinks, kernel) == plan.cost(0, n, c + n, window, sinks, kernel)
        check_items(rows, n, c, window, sinks, kernel)


@pytest.mark.parametrize("kernel", ["bf16", "fp8"])
@pytest.mark.parametrize("n,tokens", [((1 << 15) - 1, (1 << 19) - 1), (1 << 15, 1 << 19), (1 << 17, 1 << 24), (64, 1 << 24),
                                      ((1 << 18) + 33, (1 << 20) + 5), (1 << 20, 1 << 20)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100000, 40)])
def test_costs_of_long_sequences(plan, kernel, n, tokens, window, sinks):
    """Costs by the closed form against the sum of the items', and the limit below which 32 bits do."""
    rows = plan.items(1, n, tokens - n, window, sinks, kernel)
    assert int(rows[:, 0].sum()) == plan.cost(1, n, tokens, window, sinks, kernel)
    tile, item, _ = KERNELS[kernel]
    assert (rows[:, 0] == rows[:, 1] * np.array(tile)[rows[:, 2]] + np.array(item)[rows[:, 2]]).all()
    if plan.L.plan_short(n, tokens):
        assert plan.cost(1, n, tokens, window, sinks, kernel) == plan.cost(0, n, tokens, window, sinks, kernel) < 1 << 29
    else:
        assert n >= 1 << 15 or tokens >= 1 << 19


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_pieces_of_random_lines(plan, kernel):
    """Every item once, its parts in order and numbered without a gap, one cut item begun and one gone on in a CTA."""
    r = np.random.default_rng(2)
    for _ in range(300):
        rows = []
        for _ in range(int(np.exp(r.uniform(0, np.log(40))))):
            n = 1 if kernel.startswith("single") else int(np.exp(r.uniform(0, np.log(900))))
            c = int(np.exp(r.uniform(0, np.log(20000)))) * int(r.integers(0, 2))
            window = int(np.exp(r.uniform(0, np.log(3000)))) if r.random() < 0.2 else 0
            rows.append(plan.items(1, n, c, window, 0, kernel))
        rows = np.concatenate(rows)
        ctas = int(r.choice([1, 7, 152, 608]))
        got = plan.pieces(0, rows, kernel, ctas)
        assert 1 <= got <= ctas
        assert plan.pieces(1, rows, kernel, ctas) == got


def test_pieces_of_a_line_beyond_32_bits(plan):
    for kernel, n in (("bf16", 1 << 16), ("fp8", 1 << 15)):
        c = (1 << 24) - n
        rows = plan.items(1, n, c, 0, 0, kernel)
        assert int(rows[:, 0].sum()) > 1 << 32
        assert plan.pieces(1, rows, kernel) == 152
    for kernel in ("single bf16", "single fp8"):
        rows = np.concatenate([plan.items(1, 1, (1 << 24) - 1 - i, 0, 0, kernel) for i in range(1200)])
        assert int(rows[:, 0].sum()) > 1 << 32
        assert plan.pieces(1, rows, kernel, 608) == 608
