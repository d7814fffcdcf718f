"""Attention of chunks whose work is cut between CTAs: keys, queries and scores that are not finite, and bad page
ids, give what they give in one piece.  (3000 tokens are 24 key tiles a KV head, cut into several parts by either
kernel: a CTA gets at least 4 key tiles of the tile kernel's work, 3 (FP8 pages: 5) of the single tokens'.)"""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import chunk_helpers as ch
from tests import long_helpers as lh
from tests import paged_helpers as ph

pytestmark = pytest.mark.gpu

PS, HKV, HQ, D, GROUP = lh.PS, lh.HKV, lh.HQ, lh.D, lh.GROUP
KV = ["bf16", "fp8"]
# a single token alone; some, which have a kernel of their own behind the tiles'; tiles of one head, of two
SIZES = {"single": [(3000, 1)], "singles": [(3000, 1), (2990, 1)], "pair": [(3000, 64)], "heads": [(3000, 20)]}
G, DIM = 5, 17                                   # the KV head and dimension in which a key is large


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


def large_key(b, t):
    """Key t of sequence 0 in one dimension of one head: infinite; FP8 pages: 448 times 2^127, whose products with
    a query's entries of 2^-3 and more leave FP32's range, its other dimensions 0."""
    page, slot = b.bt[0, t // PS], t % PS
    if b.kv == "bf16":
        ph.pool_view(b.cache.host)[page, 0, G, slot, DIM] = lh.bf16_bits([np.inf])[0]
    else:
        codes = np.zeros(D, np.uint8)
        codes[DIM] = 0x7E
        b.cache.f8.set_row(page, 0, G, slot, codes, np.float32(2.0 ** 127))


def clear_signs(b):
    """Queries whose entry in that dimension is at least 1/2 in size, so that its sign is the score's."""
    q = b.q.clone()
    x = q[..., DIM].float()
    q[..., DIM] = torch.where(x < 0, x - 0.5, x + 0.5).to(torch.bfloat16)
    b.q.copy_(q)
    b.qf = q.double().cpu().numpy()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("t", [0, 1500, 2995])
def test_an_infinite_score_is_not_zeros(kv, sizes, t):
    """Scores of +inf: not a number, with no flag.  Of -inf: a weight of nothing, as if the token were not there."""
    b = ch.Batch(kv, SIZES[sizes], seed=61)
    clear_signs(b)
    large_key(b, t)
    b.upload().call()
    assert b.flag() == 0
    got = lh.bf16_values(b.out)
    heads = np.arange(G * GROUP, (G + 1) * GROUP)
    c, n = b.sizes[0]
    rest = np.setdiff1d(b.tokens[0], [t])
    K, V = b.cache.rows(b.bt[0], rest)
    others = np.setdiff1d(np.arange(HQ), heads)
    Kall, Vall = b.cache.rows(b.bt[0], b.tokens[0])
    if kv == "bf16":
        Kall[G] = 0                              # (that head is looked at below)
    Kall = np.where(np.isfinite(Kall), Kall, 0)
    seen_inf = seen_without = 0
    for i in list(range(0, n, 7)) + [n - 1]:
        upto = c + i + 1
        want, off = ch.attend(b.qf[i], K[:, rest < upto], V[:, rest < upto], kv)
        for h in heads:
            if b.qf[i, h, DIM] > 0:
                assert np.isnan(got[i, h]).all(), (i, h, got[i, h][:4])
                seen_inf += 1
            else:
                assert (np.abs(got[i, h] - want[h]) <= off[h]).all(), (i, h)
                seen_without += 1
        want, off = ch.attend(b.qf[i], Kall[:, :upto], Vall[:, :upto], kv)
        assert (np.abs(got[i] - want) <= off)[others].all(), i
    assert seen_inf and (seen_without or n == 1)
    b.check(rows=range(1, len(b.sizes))).close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("whole", [True, False])
def test_a_query_that_is_not_finite(kv, sizes, what, whole):
    """One head's query, all of it or one entry: its row is not a number, the other rows are what they were.  (Of the
    same token within the tolerance: the heads of a single token share the moves of their softmax's reference.)"""
    b = ch.Batch(kv, SIZES[sizes], seed=62).upload().call()
    assert b.flag() == 0
    want = b.out.clone()
    last = b.T - 1
    b.q[last, 9, slice(None) if whole else 3] = what
    b.call()
    assert b.flag() == 0
    assert torch.isnan(b.out[last, 9]).all()
    assert torch.equal(b.out[:last], want[:last])
    row = len(b.sizes) - 1
    K, V = b.cache.rows(b.bt[row], b.tokens[row])
    o, off = ch.attend(b.qf[last], K, V, kv)
    others = np.arange(HQ) != 9
    assert (np.abs(lh.bf16_values(b.out)[last] - o) <= off)[others].all()
    b.close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("infinite", [False, True])
def test_a_bad_page_is_zeros(kv, sizes, infinite):
    """... and a flag, whatever the scores are in the other parts."""
    b = ch.Batch(kv, SIZES[sizes], seed=63, spare=1)
    clear_signs(b)
    if infinite:
        large_key(b, 40)
        large_key(b, 2900)
    b.bt[0, 90] = b.cache.pages
    b.upload().call()
    assert b.flag() == pkv.PKV_DEVERR_PAGE_RANGE
    assert not b.out[:b.sizes[0][1]].float().any()
    b.check(rows=range(1, len(b.sizes))).close()
