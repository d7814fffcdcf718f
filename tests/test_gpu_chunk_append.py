"""Normed, rotated appends of many tokens against the formula in 64 bits.

Every value is rounded to FP32 (2^-24 of it), then to BF16: |got - want| is at most that, half a step of
want (2^(e - 8) for 2^e <= |want| < 2^(e + 1)) and 2^-36 of the row's largest for the arithmetic before it (two
FP32 parts).  (Where the FP32 number lies between two BF16 values, the even one is taken: half a step
alone would be too little.)  Values and codes have to be equal.

Query rows with norms have one FP32 part: their value before BF16 is off by 2^-24 for each of: the rotation's fused sum,
its second sum, 1 / sqrt (2 units in the last place: 2 * 2^-23), half of the 11 additions of squares (8 in a row,
then 3), the addition of eps and half of it, the product: below 16 * 2^-24 = 2^-20."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import long_helpers as lh
from tests import paged_helpers as ph

pytestmark = pytest.mark.gpu

PS, HKV, HQ, D = lh.PS, lh.HKV, lh.HQ, lh.D
KV = ["bf16", "fp8"]
MAX_POS = 4096


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


@pytest.fixture(scope="module")
def rope():
    return pkv.rope_table(MAX_POS, "cuda")


def bf16(x):
    return torch.tensor(np.asarray(x, np.float32)).to(torch.bfloat16)


def formula(x, w, eps, pos, axes):
    """x [n][h][64], pos [3][n]: the rows in FP64."""
    x = x.double().numpy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.double().numpy()
    axis = np.repeat([0, 1, 2], axes if axes else (32, 0, 0))
    angle = pos[axis].T * lh.THETA ** (-2.0 * np.arange(32) / D)              # [n][32]
    z = (x[..., :32] + 1j * x[..., 32:]) * np.exp(1j * angle)[:, None]
    return np.concatenate([z.real, z.imag], -1)


def rounded_once(got, want, what, before=2.0 ** -24):
    half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126))) - 8)
    off = half + before * np.abs(want) + 2.0 ** -36 * np.abs(want).max(-1, keepdims=True)
    bad = ~(np.abs(got.double().numpy() - want) <= off)
    assert not bad.any(), (what, np.argwhere(bad)[:3].tolist(), got.double().numpy()[bad][:3], want[bad][:3])


class Case:
    def __init__(self, kv, T, seed, norm=True, axes=None, pad=0, gap=0, scale=1.0, eps=1e-5):
        rng = np.random.default_rng(seed)
        self.kv, self.T, self.norm, self.axes, self.eps = kv, T, norm, axes, eps
        n = T - pad
        self.pages = -(-n // PS) + 3
        self.cache = lh.Cache(kv, self.pages).upload()
        at = rng.permutation(self.pages * PS)[:n]                              # places in no order
        self.slots = np.full(T, -1, np.int64)
        self.slots[rng.permutation(T)[:n]] = at                                # padding anywhere
        self.live = np.flatnonzero(self.slots >= 0)
        self.pos = rng.integers(0, MAX_POS, (3, T))
        self.pos[:, self.slots < 0] = -77                                      # (not looked at)

        def rows(h):
            x = rng.standard_normal((T, h + gap, D)) * np.exp(0.5 * rng.standard_normal((T, h + gap, 1))) * scale
            return bf16(x)

        self.full = {"q": rows(HQ), "k": rows(HKV), "v": rows(HKV)}
        self.q, self.k, self.v = (self.full[x][:, :h] for x, h in (("q", HQ), ("k", HKV), ("v", HKV)))
        self.qw, self.kw = (bf16(1 + 0.4 * rng.standard_normal(D)) if norm else None for _ in range(2))

    def run(self, rope, inplace=False, with_q=True, stream=None):
        d = {x: t.cuda() for x, t in self.full.items()}
        q, k, v = (d[x][:, :h] for x, h in (("q", HQ), ("k", HKV), ("v", HKV)))
        self.out = q if inplace else torch.full((self.T, HQ, D), 7.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        w = [None if x is None else x.cuda() for x in (self.qw, self.kw)]
        args = (self.cache.pool, k, k.stride(0), v, v.stride(0), q if with_q else None, q.stride(0),
                self.out if with_q else None, w[0] if with_q else None, w[1], self.eps, lh.dev(self.slots),
                lh.dev(self.pos.astype(np.int32)), self.T, self.axes, self.T, rope, MAX_POS, err, stream)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        pkv.pkv_chunk_append(*args)
        torch.cuda.synchronize()
        return int(err)

    def check(self, with_q=True, padding=7.0):
        n = self.live
        pos = self.pos[:, n]
        host = self.cache.host.copy()                                          # all NaN
        if with_q:
            got = self.out.cpu()
            rounded_once(got[n], formula(self.q[n], self.qw, self.eps, pos, self.axes), "q",
                         2.0 ** -20 if self.norm else 2.0 ** -24)
            rest = np.setdiff1d(np.arange(self.T), n)
            if padding is not None:
                assert (got[rest] == padding).all()
        want_k = formula(self.k[n], self.kw, self.eps, pos, self.axes)
        got = self.cache.download()
        page, slot = self.slots[n] // PS, self.slots[n] % PS
        if self.kv == "bf16":
            P = ph.pool_view(got.copy())
            K = torch.from_numpy(P[page, 0, :, slot].view(np.int16).copy()).view(torch.bfloat16)
            rounded_once(K, want_k, "k")
            assert np.array_equal(P[page, 1, :, slot], self.v[n].contiguous().view(torch.int16).numpy().view(np.uint16))
            P[page, :, :, slot] = ph.SENTINEL
            assert np.array_equal(P.reshape(-1), host)                         # nothing else was written
        else:
            k = torch.from_numpy(want_k).float().to(torch.bfloat16)            # (the roundings of the kernel)
            for i, t in enumerate(n):
                self.cache.put(page[i], slot[i], k[i].float().numpy(), self.v[t].float().numpy())
            assert np.array_equal(got, self.cache.host)
        self.cache.close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("axes", [None, (8, 12, 12), (32, 0, 0), (0, 1, 31)])
@pytest.mark.parametrize("T,pad,gap", [(1, 0, 0), (2, 1, 0), (7, 0, 1), (37, 5, 8), (300, 0, 3)])
def test_rows(kv, norm, axes, T, pad, gap, rope):
    c = Case(kv, T, 1000 + T, norm, axes, pad, gap)
    assert c.run(rope) == 0
    c.check()


@pytest.mark.parametrize("kv", KV)
def test_many_tokens(kv, rope):
    c = Case(kv, 2500, 5, True, (8, 12, 12), 100, 0)
    assert c.run(rope) == 0
    c.check()


@pytest.mark.parametrize("scale,eps", [(2.0 ** 100, 1e-6), (2.0 ** 120, 1e-6), (2.0 ** -60, 1e-5), (2.0 ** -10, 1e-6),
                                       (0.0, 1e-6), (2.0 ** 62, 1e-5), (2.0 ** 57, 1.0)])
def test_norms_of_large_and_small_rows(scale, eps, rope):
    c = Case("bf16", 40, 6, scale=scale, eps=eps)
    assert torch.isfinite(c.q.float()).all()
    assert c.run(rope) == 0
    c.check()


@pytest.mark.parametrize("kv", KV)
def test_in_place_and_without_queries(kv, rope):
    c = Case(kv, 50, 7, pad=8)
    assert c.run(rope, inplace=True) == 0
    rest = np.setdiff1d(np.arange(50), c.live)
    assert torch.equal(c.out.cpu()[rest], c.q[rest])
    c.check(padding=None)
    c = Case(kv, 50, 8, pad=8)
    assert c.run(rope, with_q=False) == 0
    c.check(with_q=False)


@pytest.mark.parametrize("kv", KV)
def test_without_norms_the_bits_of_a_prefill(kv, rope):
    T = 75
    c = Case(kv, T, 9, norm=False)
    table = np.random.default_rng(1).permutation(c.pages)[None, :].astype(np.int32)
    p = 5 + np.arange(T)
    c.slots, c.pos, c.live = table[0, p // PS].astype(np.int64) * PS + p % PS, np.stack([p] * 3), np.arange(T)
    assert c.run(rope) == 0
    got = c.cache.slab.clone()
    other = lh.Cache(kv, c.pages).upload()
    pkv.pkv_prefill_append(other.pool, c.k.contiguous().cuda(), c.v.contiguous().cuda(), lh.dev(table), c.pages, 1, 5, T,
                           rope, MAX_POS)
    assert torch.equal(got, other.slab)
    q = c.q.contiguous().cuda()
    pkv.pkv_append_rope(other.pool, c.k.contiguous().cuda(), c.v.contiguous().cuda(), q, lh.dev(np.repeat(table, T, 0)),
                        c.pages, lh.dev(p.astype(np.int32)), T, rope, MAX_POS)
    assert torch.equal(c.out, q) and torch.equal(other.slab, got)
    other.close()
    c.cache.close()


@pytest.mark.parametrize("kv", KV)
def test_tokens_that_are_refused_leave_everything(kv, rope):
    c = Case(kv, 40, 10, axes=(8, 12, 12))
    c.slots[3], c.slots[5], c.slots[9] = c.pages * PS, -2, 2 ** 40
    assert c.run(rope) == pkv.PKV_DEVERR_PAGE_RANGE
    c.live = np.setdiff1d(c.live, [3, 5, 9])
    c.check()
    c = Case(kv, 40, 11, axes=(8, 12, 12))
    c.pos[0, 3], c.pos[1, 5], c.pos[2, 9] = MAX_POS, -1, 2 ** 31 - 1
    assert c.run(rope) == pkv.PKV_DEVERR_LENGTH
    c.live = np.setdiff1d(c.live, [3, 5, 9])
    c.check()


def test_rows_that_are_not_finite_stay_to_themselves(rope):
    c = Case("bf16", 8, 12)
    for t in (c.full["q"], c.full["k"]):
        t[2, 1, 5], t[3, 2, 40] = float("nan"), float("inf")
    assert c.run(rope) == 0
    got = c.out.cpu()
    assert torch.isnan(got[2, 1]).all() and not torch.isfinite(got[3, 2]).all()
    page, slot = c.slots // PS, c.slots % PS
    K = torch.from_numpy(ph.pool_view(c.cache.download())[page, 0, :, slot].view(np.int16).copy()).view(torch.bfloat16)
    for x, full, w in ((got, c.q, c.qw), (K, c.k, c.kw)):
        keep = [(t, h) for t in range(8) for h in range(x.shape[1]) if (t, h) not in ((2, 1), (3, 2))]
        t, h = np.array(keep).T
        want = formula(full, w, c.eps, c.pos, None)
        rounded_once(x[t, h], want[t, h], "rows", 2.0 ** -20)
    c.cache.close()


@pytest.mark.parametrize("kv", KV)
def test_on_another_stream(kv, rope):
    c = Case(kv, 60, 13)
    assert c.run(rope, stream=torch.cuda.Stream()) == 0
    c.check()


@pytest.mark.parametrize("kv", KV)
def test_one_slot_twice_touches_nothing_else(kv, rope):
    pools = []
    for twice in (True, False):
        c = Case(kv, 40, 77)
        place = int(c.slots[0])
        c.slots[:2] = place if twice else -1
        assert c.run(rope) == 0
        c.cache.host[:] = c.cache.download()
        c.cache.put(place // PS, place % PS, np.ones((HKV, D)), np.ones((HKV, D)))
        pools.append(c.cache.host.copy())
        c.cache.close()
    assert np.array_equal(*pools)
