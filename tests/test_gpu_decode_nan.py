"""A query that is not a number, over caches long enough to be cut: its row is not a number in any of the decode calls,
and the others are what they are by themselves."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import chunk_helpers as ch
from tests import long_helpers as lh

pytestmark = pytest.mark.gpu

PS, HKV, HQ, D = lh.PS, lh.HKV, lh.HQ, lh.D
B, TOKENS, HEAD = 4, 1500, 9


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


def calls(b):
    """name -> call(out): every decode call over the batch, units of 4 pages (24 of them) and of 16 (6)."""
    pool, q, bt, blocks, lens, err = b.cache.pool, b.q, b.dev["bt"], b.blocks, b.dev["lens"], b.err
    keep = []

    def ws(nbytes):
        keep.append(torch.zeros(nbytes, dtype=torch.uint8, device="cuda"))
        return keep[-1], nbytes

    def i32(*x):
        keep.append(lh.dev(np.array(x, np.int32)))
        return keep[-1]

    for ppc in (4, 16):
        w = ws(pkv.pkv_decode_workspace_bytes(B, blocks, ppc))
        variants = dict(default=0, mma=pkv.PKV_DECODE_MMA, split=pkv.PKV_DECODE_SPLIT_MERGE)
        if b.kv == "bf16":
            variants["simt"] = pkv.PKV_DECODE_SIMT
        for name, v in variants.items():
            yield f"{name} {ppc}", lambda out, v=v, w=w, ppc=ppc: pkv.pkv_decode_attention_variant(
                pool, q, bt, blocks, lens, B, lh.SCALE, ppc, *w, out, err, None, v)
        w = ws(pkv.pkv_decode_window_workspace_bytes(B, blocks, 1400, 4, ppc))
        yield f"window {ppc}", lambda out, w=w, ppc=ppc: pkv.pkv_decode_window(
            pool, q, bt, blocks, lens, B, lh.SCALE, 1400, 4, ppc, *w, out, err)
        n = blocks * PS
        acc = [torch.zeros((B, HKV, n), device="cuda") for _ in range(2)]
        w = ws(pkv.pkv_decode_scored_workspace_bytes(B, blocks, ppc))
        yield f"scored {ppc}", lambda out, w=w, ppc=ppc, acc=acc: pkv.pkv_decode_scored(
            pool, q, bt, blocks, lens, B, lh.SCALE, *acc, n, ppc, *w, out, err)
        w = ws(pkv.pkv_decode_shared_workspace_bytes(B, blocks, 1, 64, ppc, 16))
        starts, prefix = i32(0, B), i32(64)
        yield f"shared {ppc}", lambda out, w=w, ppc=ppc: pkv.pkv_decode_shared(
            pool, q, bt, blocks, lens, B, starts, prefix, 1, 64, lh.SCALE, ppc, 16, *w, out, err)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("whole", [True, False])
def test_its_row_is_not_a_number(kv, whole):
    b = ch.Batch(kv, [(TOKENS + 3 * i, 1) for i in range(B)], seed=201)
    b.bt[1:, :64] = b.bt[0, :64]                              # (the shared call's prefix)
    b.upload()
    clean = {name: torch.full_like(b.out, ch.SENTINEL) for name, _ in calls(b)}
    for name, call in calls(b):
        call(clean[name])
    b.q[2, HEAD, slice(None) if whole else 11] = float("nan")
    others = torch.ones(HQ, dtype=torch.bool, device="cuda")
    others[HEAD // 4 * 4:HEAD // 4 * 4 + 4] = False           # (the KV head's four share what a warp does)
    for name, call in calls(b):
        out = torch.full_like(b.out, ch.SENTINEL)
        call(out)
        assert b.flag() == 0, name
        assert torch.isnan(out[2, HEAD]).all(), (name, out[2, HEAD, :4].tolist())
        rest = [0, 1, 3]
        assert torch.equal(out[rest], clean[name][rest]), name
        assert torch.equal(out[2, others], clean[name][2, others]), name
        near = clean[name][2].float()
        group = [h for h in range(HEAD // 4 * 4, HEAD // 4 * 4 + 4) if h != HEAD]
        assert (out[2, group].float() - near[group]).abs().max() <= 0.02 * near.abs().max(), name
    b.close()
