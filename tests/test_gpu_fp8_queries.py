"""Infinite queries over FP8 pages: a row that is not a number, as over BF16 pages, however small the keys are."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import chunk_helpers as ch
from tests import long_helpers as lh

pytestmark = pytest.mark.gpu

HKV, HQ, D, PS = lh.HKV, lh.HQ, lh.D, lh.PS


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("what", [float("inf"), -float("inf")])
@pytest.mark.parametrize("tokens", [40, 700])
def test_an_infinite_entry_makes_its_row_not_a_number(kv, what, tokens):
    b = ch.Batch(kv, [(tokens, 1), (17, 1), (5, 1)], seed=81)
    for row, at in enumerate(b.tokens):
        for t in at:                                        # scores of 2^-30 times an entry of the query
            k, v = b.rng.standard_normal((2, HKV, D))
            b.cache.put(b.bt[row, t // PS], t % PS, k * 2.0 ** -30, v)
    b.q[0, 9, 5] = what
    b.upload()
    B, bt, lens = 3, b.dev["bt"], b.dev["lens"]
    outs = {"chunk": b.out}
    b.call()
    one = torch.full((1, HQ, D), ch.SENTINEL, dtype=torch.bfloat16, device="cuda")
    starts = lh.dev(np.array([0, 1], np.int32))
    pkv.pkv_chunk_attention(b.cache.pool, b.q, bt, b.blocks, lens, starts, 1, 1, lh.SCALE, 0, 0, b.ws, b.nbytes, one, b.err)
    outs["one token"] = torch.cat([one, b.out[1:]])
    ws = torch.zeros(pkv.pkv_decode_workspace_bytes(B, b.blocks, 4), dtype=torch.uint8, device="cuda")
    outs["decode"] = torch.empty_like(b.out)
    pkv.pkv_decode_attention(b.cache.pool, b.q, bt, b.blocks, lens, B, lh.SCALE, 4, ws, ws.numel(), outs["decode"], b.err)
    n = b.blocks * PS
    acc = torch.zeros((B, HKV, n), device="cuda")
    gathered = torch.empty_like(acc)
    nbytes = pkv.pkv_decode_scored_workspace_bytes(B, b.blocks, 4)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    outs["scored"] = torch.empty_like(b.out)
    pkv.pkv_decode_scored(b.cache.pool, b.q, bt, b.blocks, lens, B, lh.SCALE, acc, gathered, n, 4, ws, nbytes, outs["scored"], b.err)
    assert b.flag() == 0
    K, V = b.cache.rows(b.bt[0], b.tokens[0])
    want, off = ch.attend(b.qf[0], K, V, kv)
    others = np.arange(HQ) != 9
    for name, out in outs.items():
        got = lh.bf16_values(out)
        assert np.isnan(got[0, 9]).all(), (name, got[0, 9][:4])
        assert (np.abs(got[0] - want) <= off)[others].all(), name
        b.check(rows=[1, 2], out=out)
    b.close()
