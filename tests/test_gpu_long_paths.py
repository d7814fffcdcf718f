"""Loops of the long-context kernels that small cases do not go round: a prefix CTA's later work items, groups
beyond a warp's lanes, units that a CTA takes one after another, copies of several steps, and the weights
of long rows added in the attention's own launch.  Each test first says, from the sizes that the library works
by, that its case goes there."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import long_helpers as lh
from tests import paged_helpers as ph
from tests import test_gpu_long as tl

pytestmark = pytest.mark.gpu

PS, HKV, HQ, D = lh.PS, lh.HKV, lh.HQ, lh.D
KV = ["bf16", "fp8"]
SMS = 152
native = tl.native


def random_cache(kv, pages, seed):
    """A pool of random rows: N(0, 1) with a few keys eight times as large (BF16), any finite codes with row
    scales of 0.001 to 0.01 (FP8)."""
    rng = np.random.default_rng(seed)
    c = lh.Cache(kv, pages)
    if kv == "bf16":
        P = ph.pool_view(c.host)
        for p in range(0, pages, 512):
            x = rng.standard_normal(P[p:p + 512].shape)
            x[:, 0][rng.random(x[:, 0].shape[:-1]) < 0.01] *= 8
            P[p:p + 512] = lh.bf16_bits(x)
    else:
        c.host[:] = rng.integers(0, 127, c.host.size, dtype=np.uint8) | (rng.integers(0, 2, c.host.size, dtype=np.uint8) << 7)
        c.f8.scales[...] = rng.uniform(0.001, 0.01, c.f8.scales.shape)
    return c, rng


def spoil(c, table_row, L):
    """NaN behind the last token of a sequence's last page."""
    for t in range(L, -(-L // PS) * PS):
        page, slot = table_row[t // PS], t % PS
        if c.kv == "bf16":
            ph.pool_view(c.host)[page, :, :, slot] = 0x7FFF
        else:
            for i in (0, 1):
                for h in range(HKV):
                    c.f8.set_row(page, i, h, slot, np.full(D, 0x7F, np.uint8), np.float32(np.nan))


def rows(c, table_row, n):
    """Cache.rows of the first n tokens, by the index that the cache has."""
    t = np.arange(n)
    pages, slots = np.asarray(table_row)[t // PS], t % PS
    if c.kv == "bf16":
        return c.rows(table_row, t)
    x = lh.E4M3[c.host[c.f8.index[pages, :, :, slots]]] * c.f8.scales[pages, :, :, slots].astype(np.float64)[..., None]
    return x[:, 0].transpose(1, 0, 2), x[:, 1].transpose(1, 0, 2)


def attend_gpu(q, K, V, kv, rounding=None):
    """long_helpers.attend of rows q [n][32][64] over one set of tokens K, V [8][t][64], on the device in FP64."""
    q, K, V = (torch.as_tensor(x, dtype=torch.float64, device="cuda") for x in (q, K, V))
    q = q.view(-1, HKV, 4, D).transpose(0, 1)                                  # [8][n][4][64]
    s = torch.einsum("gnhd,gtd->gnht", q, K) * lh.SCALE
    p = torch.softmax(s, -1)
    ds = lh.SCALE * 2.0 ** -18 * torch.einsum("gnhd,gtd->gnht", q.abs(), K.abs())
    if kv == "fp8":
        ds = ds + lh.SCALE * 2.0 ** -17 * q.abs().amax(-1)[..., None] * K.abs().sum(-1)[:, None, None]
    ds = ds + 2.0 ** -20 * (1 + s.abs())
    dp = p * 2 * ds.amax(-1, keepdim=True) + 2.0 ** -126
    out = torch.einsum("gnht,gtd->gnhd", p, V)
    rounding = rounding or (2.0 ** -8 if kv == "bf16" else 2.0 ** -11)
    off = torch.einsum("gnht,gtd->gnhd", p * rounding + dp, V.abs())
    if kv == "fp8":
        off = off + 2.0 ** -24 * V.abs().amax((1, 2))[:, None, None, None] * K.shape[1]
    off = off + 2.0 ** -8 * out.abs() + 2.0 ** -126
    flat = [x.transpose(0, 1).reshape(-1, HQ, D).cpu().numpy() for x in (out, off)]
    return (*flat, p.transpose(0, 1).cpu().numpy(), dp.transpose(0, 1).cpu().numpy())      # p [n][8][4][t]


def grouped(kv, groups, seed):
    """shared_case for large cases, its rows random as a whole."""
    own = [n for _, ns in groups for n in ns]
    of = [i for i, (_, ns) in enumerate(groups) for _ in ns]
    prefix = np.array([p for p, _ in groups], dtype=np.int32)
    starts = np.concatenate([[0], np.cumsum([len(ns) for _, ns in groups])]).astype(np.int32)
    pages = int(prefix.sum()) + sum(-(-n // PS) for n in own)
    blocks = max(int(prefix[g]) + -(-n // PS) for g, n in zip(of, own))
    c, rng = random_cache(kv, pages, seed)
    ids = rng.permutation(pages).astype(np.int32)
    bt = np.full((len(own), blocks), -1, dtype=np.int32)
    view, at = bt.copy(), 0
    for g, (p, ns) in enumerate(groups):
        row = ids[at:at + p]
        at += p
        bt[starts[g], :p] = row
        for b in range(starts[g], starts[g + 1]):
            n = -(-own[b] // PS)
            view[b, :p] = row
            bt[b, p:p + n] = view[b, p:p + n] = ids[at:at + n]
            at += n
            spoil(c, view[b], int(p) * PS + own[b])
    lens = np.array([prefix[g] * PS + n for g, n in zip(of, own)], dtype=np.int32)
    return c.upload(), bt, view, lens, starts, prefix, rng


def check_shared(c, kv, view, lens, starts, prefix, qf, outs):
    for g in range(len(prefix)):
        for b in range(starts[g], starts[g + 1]):
            K, V = rows(c, view[b], int(lens[b]))
            want, off, _, _ = attend_gpu(qf[b][None], K, V, kv, 2.0 ** -8)
            for o in outs:
                tl.close(o[b], want[0], off[0], (b, int(lens[b])))


def prefix_items(groups, chunk_pages):
    """Work items of the prefix kernel: a group's row tiles of 32 sequences in pairs, each pair in every chunk, an odd
    last tile in two chunks at a time, for each KV head."""
    n = 0
    for p, ns in groups:
        tiles, chunks = -(-len(ns) // 32), -(-p // chunk_pages)
        n += HKV * (tiles // 2 * chunks + tiles % 2 * -(-chunks // 2))
    return n


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("groups", [
    # two pairs and an odd tile; one odd tile whose last item has no second chunk; a pair and an odd tile
    [(130, [1 + i % 20 for i in range(130)]), (133, [5, 33, 2]), (40, [7] * 70)],
    # odd tiles alone: every item is two chunks of one tile, many CTAs have a last one with one
    [(129, [3 + 5 * i for i in range(9)]), (97, [20] * 32), (121, [1]), (137, [4, 50])],
])
def test_prefix_ctas_with_several_items(kv, groups):
    items = prefix_items(groups, 8)
    assert items > SMS * 3 // 2 and items % SMS and any(-(-p // 8) % 2 for p, _ in groups)
    c, bt, view, lens, starts, prefix, rng = grouped(kv, groups, 500)
    q, qf = lh.query(rng, len(lens))
    outs = [tl.run_shared(c, bt, lens, starts, prefix, q, *a)[0] for a in ((0, 8), (3, 8), (0, 0))]
    check_shared(c, kv, view, lens, starts, prefix, qf, outs)
    # the same bits again, launch behind launch, and with scores that move the references
    again = tl.run_shared(c, bt, lens, starts, prefix, q, 3, 8)[0]
    assert torch.equal(outs[1], again)
    far, farf = q * 256, qf * 256
    check_shared(c, kv, view, lens, starts, prefix, farf, [tl.run_shared(c, bt, lens, starts, prefix, far, 3, 8)[0]])
    c.close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("count", [33, 100])
def test_more_groups_than_lanes(kv, count):
    """Groups beyond the 32 that a warp holds at once, some without a prefix."""
    rng = np.random.default_rng(9)
    groups = [(int(rng.integers(0, 4)) * int(rng.integers(1, 6)), [int(n) for n in rng.integers(0, 40, rng.integers(1, 4))])
              for _ in range(count)]
    groups = [(p, [n + (p == 0) for n in ns]) for p, ns in groups]            # (a sequence has a token)
    groups[-1], groups[32] = (11, [40, 0, 3]), (9, [7])
    assert len(groups) > 32 and any(p == 0 for p, _ in groups[:32]) and any(p == 0 for p, _ in groups[32:]) or count == 33
    assert count == 33 or prefix_items(groups, 8) > SMS
    c, bt, view, lens, starts, prefix, rng = grouped(kv, groups, 510)
    q, qf = lh.query(rng, len(lens))
    outs = [tl.run_shared(c, bt, lens, starts, prefix, q, *a)[0] for a in ((0, 0), (2, 8), (1, 16))]
    check_shared(c, kv, view, lens, starts, prefix, qf, outs)
    c.close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("batch,first", [(260, 9), (19, 9), (19, 0)])
def test_ctas_with_several_units(kv, batch, first):
    """Own pages in chunks of one page, more of them than CTAs a (sequence, KV head): a CTA goes on to its next chunk
    with its barriers made anew.  260 sequences: a third launch merges; 19: the units do; without a prefix: the units
    alone."""
    rng = np.random.default_rng(11)
    own = [int(n) for n in rng.integers(1, 60, batch)]
    for b in (0, 7, batch - 1):
        own[b] = int(rng.integers(450, 640))
    ctas = max(1, SMS * 16 // (batch * HKV))
    assert -(-max(own) // PS) > ctas
    c, bt, view, lens, starts, prefix, rng = grouped(kv, [(first, own)], 520)
    q, qf = lh.query(rng, batch)
    outs = []
    for ring in (0, 2, 3, 4):
        outs.append(tl.run_shared(c, bt, lens, starts, prefix, q, 1, 8, pkv.PKV_STEP_RING(ring) if ring else 0)[0])
        assert torch.equal(outs[-1], outs[0])
    outs.append(tl.run_shared(c, bt, lens, starts, prefix, q, 5, 8)[0])
    check_shared(c, kv, view, lens, starts, prefix, qf, [outs[0], outs[-1]])
    c.close()


@pytest.mark.parametrize("kv", KV)
def test_evict_copies_of_several_steps(kv):
    """Copy warps that go on to their next 32 tokens, whose rows they have looked up meanwhile."""
    rng = np.random.default_rng(12)
    B, keep, recent, sinks = 64, 1000, 100, 4
    lens = np.concatenate([rng.integers(0, 1600, B - 6), [1000, 1001, 31, 33, 64, 0]]).astype(np.int32)
    need, dneed = -(-lens // PS), -(-np.minimum(lens, keep) // PS)
    steps = -(-keep // 32)
    assert min(8, -(-steps * B // (SMS * 8))) >= 2
    bt, n = lh.shuffled_tables(rng, need, int(need.max()))
    dst, m = lh.shuffled_tables(rng, dneed, int(dneed.max()), n)
    c = lh.Cache(kv, n + m)
    c.host[:] = rng.integers(0, 256, c.host.nbytes, dtype=np.uint8).view(c.host.dtype)
    c.upload()
    acc = tl.acc_of(rng, (B, HKV, bt.shape[1] * PS), "real")
    acc_out, kept, lens_out, _ = tl.run_evict(c, bt, lens, dst, acc, keep, recent, sinks)
    want = c.host.copy()
    P, W = (ph.pool_view(x) if kv == "bf16" else ph.Fp8Pages(x) for x in (c.host, want))
    for b, L in enumerate(lens):
        nk = min(int(L), keep)
        assert lens_out[b] == nk
        for g in range(HKV):
            ids = np.array(tl.plain_evict(acc[b, g], int(L), keep, recent, sinks), np.int64)
            assert np.array_equal(kept[b, g, :nk], ids) and (kept[b, g, nk:] == -1).all()
            assert np.array_equal(acc_out[b, g, :nk], acc[b, g, ids]) and not acc_out[b, g, nk:].any()
            at = np.arange(nk)
            src, ss, dp, ds = bt[b][ids // PS], ids % PS, dst[b][at // PS], at % PS
            if kv == "bf16":
                W[dp, :, g, ds] = P[src, :, g, ss]
            else:
                W.pool[W.index[dp, :, g, ds]] = c.host[P.index[src, :, g, ss]]
                W.scales.view(np.uint32)[dp, :, g, ds] = P.scales.view(np.uint32)[src, :, g, ss]
    assert np.array_equal(c.download().view(np.uint8), want.view(np.uint8))       # nothing else has changed
    c.close()


@pytest.mark.parametrize("kv", KV)
def test_weights_of_long_rows_in_the_attentions_launch(kv):
    """Rows over 2048 tokens of 57 sequences and more have their weights added by the units that finish them; and
    the library's own units are dispatched largest first."""
    rng = np.random.default_rng(13)
    B, blocks = 64, 300
    lens = rng.integers(1, 90, B).astype(np.int32)
    lens[[0, 5, 63]] = [4800, 2111, 4097]
    chunks = max(1, SMS * 6 * 2 // (B * HKV))
    units = (-(-blocks // chunks) + 3) // 4 * 4
    assert B * HKV >= 3 * SMS and 2048 < blocks * PS <= 16384
    assert units > 64 and B * HKV * -(-blocks // units) > SMS * 6
    need = -(-lens // PS)
    c, rng = random_cache(kv, int(need.sum()), 530)
    bt, _ = lh.shuffled_tables(rng, need, blocks)
    for b, L in enumerate(lens):
        spoil(c, bt[b], int(L))
    c.upload()
    q, qf = lh.query(rng, B)
    a0 = rng.random((B, HKV, blocks * PS)).astype(np.float32)
    got = []
    for ppc in (0, units, 7):
        acc, acc_out = lh.dev(a0), torch.full((B, HKV, blocks * PS), -9.0, device="cuda")
        out, _ = tl.run_scored(c, bt, lens, q, acc, acc_out, ppc)
        got.append((out, acc_out))
        assert np.array_equal(acc.cpu().numpy(), a0)
    # the same units, dispatched in another order
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    for b, L in enumerate(lens):
        K, V = rows(c, bt[b], int(L))
        want, off, p, dp = attend_gpu(qf[b][None], K, V, kv)
        p, dp = p[0].sum(1), dp[0].sum(1)
        w = a0[b, :, :L] + p
        for out, acc_out in got:
            tl.close(out[b], want[0], off[0], (b, int(L)))
            x = acc_out[b].cpu().numpy().astype(np.float64)
            assert (np.abs(x[:, :L] - w) <= dp + 2.0 ** -20 * p + 2.0 ** -24 * 4 * w).all(), b
            assert (x[:, L:] == -9.0).all()
    c.close()
