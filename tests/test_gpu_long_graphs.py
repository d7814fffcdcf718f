"""Captured graphs of an engine that goes on being used: what a graph holds the address of stays."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from paged_kv_decode_12_gb300.engine import DecodeEngine
from tests import long_helpers as lh
from tests import test_gpu_long as tl

pytestmark = pytest.mark.gpu

native = tl.native


@pytest.mark.parametrize("kv", tl.KV)
def test_a_captured_call_outlives_a_larger_one(kv):
    """attention_shared with a short prefix is captured, then called with a longer one (a larger
    workspace); whatever memory comes free is filled; the graph still gives what it gave."""
    c, bt, view, lens, starts, prefix, rng = tl.shared_case(kv, [(9, [20, 5, 33]), (2, [7, 40])], 31, extra_blocks=300)
    B = lens.size
    eng = DecodeEngine(c.pages, 1, B, max_blocks=bt.shape[1], pages_per_chunk=4, kv=kv)
    eng.slab.copy_(c.slab)
    eng.set_tables(bt[None])
    q, qf = lh.query(rng, B)
    args = (0, q, lh.dev(lens), lh.dev(starts), lh.dev(prefix))
    want, out = torch.empty_like(q), torch.empty_like(q)
    eng.attention_shared(*args, 9, want, prefix_pages_per_chunk=8)
    held = eng._extra_ws["shared"][-1].numel()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            eng.attention_shared(*args, 9, out, prefix_pages_per_chunk=8)
    larger = torch.empty_like(q)
    eng.attention_shared(*args, 300, larger, prefix_pages_per_chunk=8)
    assert eng._extra_ws["shared"][-1].numel() > held
    fresh = [torch.full((held,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    assert torch.equal(larger, want)             # (fixed chunks: the bound on the prefixes changes no bit)
    assert all(bool((t == 0x5A).all()) for t in fresh)
    assert eng.check_errors() == (pkv.PKV_OK, 0)
    for b in range(B):
        K, V = c.rows(view[b], range(int(lens[b])))
        tl.close(out[b], *lh.attend(qf[b], K, V, kv, 2.0 ** -8)[:2])
    eng.close()
    c.close()


@pytest.mark.parametrize("kv", tl.KV)
def test_a_captured_call_reads_the_tables_that_are_set(kv):
    """The same cache held twice, on other pages and in other rows' order: the graph follows the tables."""
    c, bt, lens, rng = tl.whole_case(kv, [100, 100, 100], 61)
    B, blocks = bt.shape
    eng = DecodeEngine(c.pages, 1, B, max_blocks=blocks, pages_per_chunk=3, kv=kv)
    eng.slab.copy_(c.slab)
    eng.set_tables(bt[None])
    q, qf = lh.query(rng, B)
    lens_d, out = lh.dev(lens), torch.empty_like(q)
    eng.attention(0, q, lens_d, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        eng.attention(0, q, lens_d, out)
    for order in ([0, 1, 2], [2, 0, 1], [1, 1, 0]):
        eng.set_tables(bt[order][None])
        fresh = [torch.full((B * blocks,), -1, dtype=torch.int32, device="cuda") for _ in range(8)]
        out.zero_()
        g.replay()
        assert eng.check_errors() == (pkv.PKV_OK, 0)
        for b in range(B):
            K, V = c.rows(bt[order[b]], range(100))
            tl.close(out[b], *lh.attend(qf[b], K, V, kv)[:2])
        assert all(bool((t == -1).all()) for t in fresh)
    eng.close()
    c.close()


@pytest.mark.parametrize("kv", tl.KV)
def test_attention_behind_an_eviction_with_a_call_elsewhere_between(kv):
    """An eviction on one stream, a call over another cache on a second one, then attention over the cut
    cache right behind the eviction: it reads the rows that the eviction has put there."""
    c, bt, lens, rng = tl.whole_case(kv, [1500, 1490, 1480, 1470], 62, blocks=100)
    B, blocks, keep = bt.shape[0], bt.shape[1], 1024
    acc = tl.acc_of(rng, (B, lh.HKV, blocks * lh.PS), "real")
    dst = np.full((B, blocks), -1, dtype=np.int32)
    dst[:, :keep // lh.PS] = np.arange(B * keep // lh.PS).reshape(B, -1)
    big = lh.Cache(kv, c.pages + B * keep // lh.PS)
    big.host[:c.host.size] = c.host
    dst[dst >= 0] += c.pages
    big.upload()
    other, obt, olens, _ = tl.whole_case(kv, [90, 33], 63)
    q, _ = lh.query(rng, B)
    n = pkv.pkv_decode_workspace_bytes(B, blocks, 16)
    ws, ws2, err = tl.ws_of(n), tl.ws_of(n), tl.flag()
    bt_d, dst_d, lens_d, acc_d = lh.dev(bt), lh.dev(dst), lh.dev(lens), lh.dev(acc)
    after, cut = torch.zeros_like(lens_d), torch.full_like(lens_d, keep)
    acc_out = torch.zeros((B, lh.HKV, blocks * lh.PS), device="cuda")
    kept = torch.zeros((B, lh.HKV, keep), dtype=torch.int32, device="cuda")
    want, out, side = (torch.empty_like(q) for _ in range(3))
    obt_d, olens_d = lh.dev(obt), lh.dev(olens)
    start = big.slab.clone()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()

    def evict(st):
        pkv.pkv_evict(big.pool, bt_d, blocks, lens_d, B, dst_d, blocks, keep, 100, 4, acc_d, acc.shape[-1], acc_out,
                      acc.shape[-1], kept, after, None, 0, err, st)

    def attend(o, st):
        pkv.pkv_decode_attention(big.pool, q, dst_d, blocks, cut, B, lh.SCALE, 16, ws, n, o, err, st)

    evict(None)
    torch.cuda.synchronize()
    attend(want, None)
    assert not torch.isnan(want).any()
    for _ in range(20):
        big.slab.copy_(start)                    # the pages to be cut to hold NaN again
        out.fill_(7.0)
        torch.cuda.synchronize()
        evict(a)
        pkv.pkv_decode_attention(big.pool, q[:2], obt_d, obt.shape[1], olens_d, 2, lh.SCALE, 16, ws2, n, side[:2], err, b)
        attend(out, a)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert pkv.pkv_check_device_error(err) == (pkv.PKV_OK, 0)
    for x in (big, c, other):
        x.close()
