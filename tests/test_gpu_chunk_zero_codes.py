"""Zeros with a sign, and rows that are not finite, quantized as the other appends do it."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import long_helpers as lh

pytestmark = pytest.mark.gpu

PS, HKV, HQ, D = lh.PS, lh.HKV, lh.HQ, lh.D


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [3, 40])
def test_they_have_the_bits_of_a_prefill(kv, T):
    gen = torch.Generator().manual_seed(T)
    k, v = torch.randn((2, T, HKV, D), generator=gen).to(torch.bfloat16)
    for x in (k, v):
        x[torch.rand(x.shape, generator=gen) < 0.3] = -0.0
        x[torch.rand(x.shape, generator=gen) < 0.1] = 0.0
        x[1, 2] = -0.0                                     # a row of nothing
        x[2, 3] = -torch.finfo(torch.bfloat16).tiny
        x[2, 4, :5] = torch.tensor([2.0 ** 100, -2.0 ** -100, -0.0, 1.0, -2.0 ** 90])
        x[0, 5, 3], x[0, 6, 2], x[0, 7, 60] = float("inf"), float("nan"), -float("inf")
    k, v = k.cuda(), v.cuda()
    pages = -(-T // PS)
    table = lh.dev(np.arange(pages)[None, :].astype(np.int32))
    slots = torch.arange(T, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rope = pkv.rope_table(64, "cuda")
    a, b = (lh.Cache(kv, pages).upload() for _ in range(2))
    pkv.pkv_chunk_append(a.pool, k, 512, v, 512, None, 0, None, None, None, 0.0, slots, pos, 0, None, T, rope, 64)
    pkv.pkv_prefill_append(b.pool, k, v, table, pages, 1, 0, T, rope, 64)
    torch.cuda.synchronize()
    assert torch.equal(a.slab, b.slab)
    a.close()
    b.close()
