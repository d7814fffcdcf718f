"""Chunks and evictions with room in turns, through the engine: the pool does not run out, and what the pages hold
stays what it was."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import chunk_helpers as ch
from tests import long_helpers as lh
from tests import test_gpu_long as tl
from tests.test_gpu_chunk_engine import Steps
from tests.test_gpu_long_engine import rows_of

pytestmark = pytest.mark.gpu

native = tl.native
PS, HKV = lh.PS, lh.HKV


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_in_turns(kv):
    s = Steps(kv, 3, layers=2, pages=60, blocks=10, T=64)
    e, rng = s.eng, np.random.default_rng(5)
    # what is neither in a table nor in the list is free, whenever nothing is behind the sequences but their room
    total = pkv.pkv_pool_info(e.pool)["num_free"] + s.pages.numel()
    for cycle in range(8):
        s.fill([20, 1, 30])
        s.launch()
        torch.cuda.synchronize()
        assert e.check_errors() == (pkv.PKV_OK, 0)
        e.read_tables()
        s.cached = s.cached + s.new
        at = 0
        for b in range(3):
            for l in range(2):
                K, V = rows_of(e, kv, l, b, range(s.cached[b]))
                i = s.new[b] - 1
                q = lh.bf16_values(s.q_out[l, at + i])
                o, off = ch.attend(q, K, V, kv)
                assert (np.abs(lh.bf16_values(s.out[l, at + i]) - o) <= off).all(), (cycle, b, l)
            at += s.new[b]
        lens = s.cached.astype(np.int32)
        acc = torch.from_numpy(rng.random((2, 3, HKV, 10 * PS)).astype(np.float32)).cuda()
        weights = acc.cpu().numpy()
        for l in range(2):
            before = [rows_of(e, kv, l, b, range(lens[b])) for b in range(3)]
            after = e.evict(l, lens, acc[l], 40, 6, 2, room=50)
            for b in range(3):
                K, V = rows_of(e, kv, l, b, range(after[b]))
                for g in range(HKV):
                    ids = tl.plain_evict(weights[l, b, g], int(lens[b]), 40, 6, 2)
                    assert np.array_equal(K[g], before[b][0][g, ids]) and np.array_equal(V[g], before[b][1][g, ids])
        s.cached = after.astype(int)
        s.lens_dev.copy_(lh.dev(after))
        named = e.bt_host[e.bt_host >= 0]
        left = s.pages.numel() - int(s.used)
        assert np.unique(named).size == named.size
        assert pkv.pkv_pool_info(e.pool)["num_free"] == total - left - named.size, cycle
        # a new list for what has been used
        pkv.pkv_pool_free(e.pool, s.pages[int(s.used):].cpu().numpy())
        s.pages.copy_(e.take_pages(s.pages.numel()))
        s.used.zero_()
    e.close()
