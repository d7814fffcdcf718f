"""The library's own unit sizes (pages_per_chunk = 0) through the engine."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from paged_kv_decode_12_gb300.engine import DecodeEngine
from tests import long_helpers as lh
from tests import test_gpu_long as tl
from tests import test_gpu_long_engine as te

pytestmark = pytest.mark.gpu

native = tl.native


@pytest.mark.parametrize("kv", tl.KV)
@pytest.mark.parametrize("fused,chains", [(True, 1), (True, 3), (False, 2)])
def test_window_engine_with_the_librarys_units(kv, fused, chains):
    layers, window, sinks, blocks = 2, 700, 5, 80
    lens = np.array([1200, 40, 997, 16, 1100, 3], dtype=np.int32)
    B = lens.size
    eng = DecodeEngine(layers * 400, layers, B, max_blocks=blocks, pages_per_chunk=0, max_pos=2048, kv=kv, fused=fused,
                       chains=chains, window=window, sinks=sinks)
    gen = torch.Generator("cuda").manual_seed(3)
    if kv == "bf16":
        eng.pool_view().copy_(torch.randn(eng.pool_view().shape, generator=gen, device="cuda"))
    else:
        codes, scales = eng.fp8_views()
        codes.copy_(torch.randint(0, 120, codes.shape, generator=gen, device="cuda", dtype=torch.uint8))
        scales.copy_(torch.rand(scales.shape, generator=gen, device="cuda") * 0.01)
    eng.build_tables(lens)
    rng = np.random.default_rng(6)
    q = te.bf16_dev(rng, (layers, B, lh.HQ, lh.D))
    kn, vn = te.bf16_dev(rng, (layers, B, lh.HKV, lh.D)), te.bf16_dev(rng, (layers, B, lh.HKV, lh.D))
    out = torch.empty_like(q)
    eng.step(q, kn, vn, lh.dev(lens - 1), lh.dev(lens), out)
    assert eng.check_errors() == (pkv.PKV_OK, 0)
    for layer in range(layers):
        for b in range(B):
            K, V = te.rows_of(eng, kv, layer, b, tl.visible(int(lens[b]), window, sinks))
            tl.close(out[layer, b], *lh.attend(lh.bf16_values(q[layer, b]), K, V, kv)[:2], (layer, b))
    # one chain: the call that a user makes without the engine
    if chains == 1:
        for layer in range(layers):
            n = pkv.pkv_decode_window_workspace_bytes(B, blocks, window, sinks, 0)
            want = torch.empty_like(out[layer])
            pkv.pkv_decode_window(eng.pool, q[layer], eng.bt[layer], blocks, lh.dev(lens), B, eng.scale, window, sinks, 0,
                                  tl.ws_of(n), n, want, eng.err)
            assert torch.equal(out[layer], want)
    eng.close()


@pytest.mark.parametrize("kv", tl.KV)
@pytest.mark.parametrize("ppc", [None, 0, 2])
def test_units_of_the_shared_and_scored_calls(kv, ppc):
    c, bt, view, lens, starts, prefix, rng = tl.shared_case(kv, [(9, [20, 5, 133]), (2, [7, 40])], 31)
    B, blocks = bt.shape
    eng = DecodeEngine(c.pages, 1, B, max_blocks=blocks, pages_per_chunk=4, kv=kv)
    eng.slab.copy_(c.slab)
    eng.set_tables(bt[None])
    q, _ = lh.query(rng, B)
    out = torch.empty_like(q)
    kw = {} if ppc is None else {"pages_per_chunk": ppc}
    eng.attention_shared(0, q, lh.dev(lens), lh.dev(starts), lh.dev(prefix), 9, out, **kw)
    assert torch.equal(out, tl.run_shared(c, bt, lens, starts, prefix, q, 4 if ppc is None else ppc, 0)[0])
    eng.set_tables(view[None])
    acc = torch.zeros((B, lh.HKV, blocks * lh.PS), device="cuda")
    want_acc = acc.clone()
    eng.attention_scored(0, q, lh.dev(lens), acc, acc, out, **kw)
    want, _ = tl.run_scored(c, view, lens, q, want_acc, want_acc, 4 if ppc is None else ppc)
    assert torch.equal(out, want) and torch.equal(acc, want_acc)
    assert eng.check_errors() == (pkv.PKV_OK, 0)
    eng.close()
    c.close()
