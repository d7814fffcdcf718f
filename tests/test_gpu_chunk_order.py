"""Chunks and single tokens right behind the kernels that make their lengths, tables, pages and queries, call after
call without a wait between: what the single tokens' kernel reads, it reads behind all of them."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import chunk_helpers as ch
from tests import long_helpers as lh

pytestmark = pytest.mark.gpu

PS, HKV, HQ, D = lh.PS, lh.HKV, lh.HQ, lh.D
B, T, BLOCKS, CALLS = 40, 160, 24, 60


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


class Run:
    """Calls of tables, append and attention, each with other counts and rows."""

    def __init__(self, kv, options):
        self.options, gen = options, torch.Generator("cuda").manual_seed(91)
        rng = np.random.default_rng(91)
        page = pkv.PKV_PAGE_BYTES if kv == "bf16" else pkv.PKV_PAGE_BYTES_FP8
        pages = B * BLOCKS
        self.slab = torch.zeros(pages * page, dtype=torch.uint8, device="cuda")
        make = pkv.pkv_pool_create if kv == "bf16" else pkv.pkv_pool_create_fp8
        self.pool = make(self.slab, self.slab.numel())
        i32 = dict(dtype=torch.int32, device="cuda")
        self.pages = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda()
        self.bt = torch.full((1, B, BLOCKS), -1, **i32)
        self.lens, self.used, self.starts = torch.zeros(B, **i32), torch.zeros(1, **i32), torch.zeros(B + 1, **i32)
        self.pos, self.err = torch.zeros(T, **i32), torch.zeros(1, **i32)
        self.slots = torch.zeros((1, T), dtype=torch.int64, device="cuda")
        self.rope = pkv.rope_table(BLOCKS * PS, "cuda")
        new = np.ones((CALLS, B), np.int32)                      # most bring one token, some a chunk or nothing
        for i in range(CALLS):
            at = rng.permutation(B)
            new[i, at[:2]] = rng.integers(2, 40, 2)
            new[i, at[2:6]] = 0
        assert new.sum(0).max() <= BLOCKS * PS and new.sum(1).max() <= T
        self.new = torch.from_numpy(new).cuda()
        self.q = torch.randn((CALLS, T, HQ, D), generator=gen, device="cuda").to(torch.bfloat16)
        self.kv = torch.randn((CALLS, 2, T, HKV, D), generator=gen, device="cuda").to(torch.bfloat16)
        self.q_out, self.out = torch.zeros_like(self.q[0]), torch.full_like(self.q, ch.SENTINEL)
        self.nbytes = pkv.pkv_chunk_attention_workspace_bytes(B, T)
        self.ws = torch.zeros(self.nbytes, dtype=torch.uint8, device="cuda")
        self.tables_ws = torch.zeros(pkv.pkv_chunk_tables_workspace_bytes(B), dtype=torch.uint8, device="cuda")

    def go(self, wait):
        for i in range(CALLS):
            pkv.pkv_chunk_tables(self.pool, self.lens, self.new[i], B, self.bt, BLOCKS, 1, self.pages, self.pages.numel(),
                                 self.used, self.used, T, self.starts, self.lens, self.pos, self.slots, self.tables_ws,
                                 self.tables_ws.numel(), self.err)
            pkv.pkv_chunk_append(self.pool, self.kv[i, 0], 512, self.kv[i, 1], 512, self.q[i], 2048, self.q_out, None, None,
                                 0.0, self.slots[0], self.pos, T, None, T, self.rope, BLOCKS * PS, self.err)
            if wait:
                torch.cuda.synchronize()
            pkv.pkv_chunk_attention(self.pool, self.q_out, self.bt[0], BLOCKS, self.lens, self.starts, B, T, lh.SCALE, 0, 0,
                                    self.ws, self.nbytes, self.out[i], self.err, None, self.options)
            if wait:
                torch.cuda.synchronize()
        return self


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("captured", [False, True])
def test_call_after_call(kv, captured):
    want = Run(kv, pkv.PKV_STEP_NO_PDL).go(True)
    got = Run(kv, 0)
    if captured:
        got.go(False)                                            # (kernels set up outside the capture)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.go(False)
        for _ in range(3):
            for x in (got.lens, got.used, got.slab):
                x.zero_()
            got.bt.fill_(-1)
            got.out.fill_(ch.SENTINEL)
            g.replay()
    else:
        got.go(False)
    torch.cuda.synchronize()
    assert int(want.err) == int(got.err) == 0
    assert torch.equal(got.lens, want.lens) and torch.equal(got.bt, want.bt)
    assert torch.equal(got.slab, want.slab)
    assert torch.equal(got.out, want.out)
    # the counters in front of the workspace's partials: (152 CTAs, 2 each), and what one kernel tells the other
    counters = 4 * (152 * 2 + 1)
    assert not want.ws[:counters].any() and not got.ws[:counters].any()
    for r in (want, got):
        pkv.pkv_pool_destroy(r.pool)
