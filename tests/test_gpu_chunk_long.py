"""Attention of chunks whose work is beyond what 32 bits count: a line of 2^30 units and more (about a second of one
GPU), sequences of 2^19 tokens and 2^15 new ones and more.

The bound is that of ``chunk_helpers.attend``, on the GPU.  Queries are 6
times a standard normal one, so that a few of the million tokens that are not the same for any two rows have all the
weight, and a row that met other tokens would be off by its whole size."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import chunk_helpers as ch
from tests import long_helpers as lh

pytestmark = pytest.mark.gpu

PS, HKV, HQ, D = lh.PS, lh.HKV, lh.HQ, lh.D
UNIT = 2 * PS * (D + 4)


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


def filled(pages, gen):
    """An FP8 pool of standard normal rows, quantized by the append."""
    slab = torch.empty(pages * pkv.PKV_PAGE_BYTES_FP8, dtype=torch.uint8, device="cuda")
    pool = pkv.pkv_pool_create_fp8(slab, slab.numel())
    rope, step = pkv.rope_table(16, "cuda"), 1 << 18
    for at in range(0, pages * PS, step):
        n = min(step, pages * PS - at)
        k, v = torch.randn((2, n, HKV, D), generator=gen, device="cuda").to(torch.bfloat16)
        pkv.pkv_chunk_append(pool, k, 512, v, 512, None, 0, None, None, None, 0.0, at + torch.arange(n, device="cuda"),
                             torch.zeros(n, dtype=torch.int32, device="cuda"), 0, None, n, rope, 16)
    return slab, pool


def rows_of_head(slab, pages, g, L):
    """K, V [L][64] in FP64 of one KV head of a sequence with the given pages."""
    u = slab.view(-1, HKV, UNIT)[pages, g]
    scales = u[:, 2 * PS * D:].contiguous().view(torch.float32).view(-1, 2, PS, 1).double()
    s, d = np.arange(PS)[:, None], np.arange(D)[None, :]
    off = (s // 2) * 2 * D + ((d // 8) ^ ((2 * (s // 2)) % 8)) * 16 + (d % 8) * 2 + s % 2
    v = u[:, PS * D + torch.from_numpy(off.reshape(-1)).cuda()]
    for x, i in ((u[:, :PS * D], 0), (v, 1)):
        x = x.contiguous().view(torch.float8_e4m3fn).double().view(-1, PS, D) * scales[:, i]
        yield x.view(-1, D)[:L]


def check(q, out, slab, pages, L, rows, positions, heads):
    for h in heads:
        K, V = rows_of_head(slab, pages, h // 4, L)
        for t, p in zip(rows, positions):
            x = q[t, h].double()
            s = K[:p + 1] @ x * lh.SCALE
            ds = lh.SCALE * (2.0 ** -18 * float((K[:p + 1].abs() @ x.abs()).max()) +
                             2.0 ** -17 * float(x.abs().max()) * float(K[:p + 1].abs().sum(-1).max()))
            ds += 2.0 ** -20 * (1 + float(s.abs().max()))
            w = torch.softmax(s, -1)
            want, mass = w @ V[:p + 1], w @ V[:p + 1].abs()
            off = (2.0 ** -8 + 2 * ds) * mass + 2 * 2.0 ** -8 * want.abs() + 2.0 ** -20
            assert float(want.abs().max()) > 16 * float(off.max())            # (the rows say something)
            bad = ~((out[t, h].double() - want).abs() <= off)
            assert not bad.any(), (t, h, bad.nonzero()[:4].tolist())
        del K, V


def test_one_long_prompt_behind_a_longer_one():
    """2^15 new tokens behind 2.4 million: 1.02 x 2^30 units."""
    n, L = 1 << 15, (1 << 21) + 370000
    gen = torch.Generator("cuda").manual_seed(1)
    need = -(-L // PS)
    slab, pool = filled(need, gen)
    bt = torch.randperm(need, generator=gen, device="cuda").to(torch.int32)
    q = (6 * torch.randn((n, HQ, D), generator=gen, device="cuda")).to(torch.bfloat16)
    out = torch.full_like(q, ch.SENTINEL)
    nbytes = pkv.pkv_chunk_attention_workspace_bytes(1, n)
    ws, err = torch.zeros(nbytes, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.pkv_chunk_attention(pool, q, bt, need, lh.dev(np.array([L], np.int32)), lh.dev(np.array([0, n], np.int32)), 1, n,
                            lh.SCALE, 0, 0, ws, nbytes, out, err)
    assert int(err) == 0
    assert not (out == ch.SENTINEL).all(-1).any()
    rows = [0, 1, 63, 64, 4095, 10000, 16384, 20011, 32703, 32704, n - 1]
    check(q, out, slab, bt.long(), L, rows, [L - n + t for t in rows], (0, 13, 31))
    # the counters are as they were
    assert not ws[:4 * 305].any()
    pkv.pkv_pool_destroy(pool)


def test_many_long_sequences_of_one_token():
    """4096 sequences that share the pages of a million tokens: 1.02 x 2^30 units."""
    B, L = 4096, (1 << 20) + 20000
    gen = torch.Generator("cuda").manual_seed(2)
    need = -(-L // PS)
    slab, pool = filled(need, gen)
    order = torch.randperm(need, generator=gen, device="cuda").to(torch.int32)
    bt = order.expand(B, need).contiguous()
    lens = (L - torch.arange(B, device="cuda") % 5).to(torch.int32)
    q = (6 * torch.randn((B, HQ, D), generator=gen, device="cuda")).to(torch.bfloat16)
    out = torch.full_like(q, ch.SENTINEL)
    nbytes = pkv.pkv_chunk_attention_workspace_bytes(B, B)
    ws, err = torch.zeros(nbytes, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    pkv.pkv_chunk_attention(pool, q, bt, need, lens, starts, B, B, lh.SCALE, 0, 0, ws, nbytes, out, err)
    assert int(err) == 0
    assert not (out == ch.SENTINEL).all(-1).any()
    rows = [0, 1, 700, 2047, 3333, B - 1]
    check(q, out, slab, order.long(), L, rows, [L - t % 5 - 1 for t in rows], (0, 13, 31))
    pkv.pkv_pool_destroy(pool)
