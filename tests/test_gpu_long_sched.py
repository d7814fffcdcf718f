"""Evictions beside a scheduler: the pages of its requests are refused, with nothing done."""
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
def test_evictions_refuse_what_is_not_the_callers(kv):
    blocks, lens = 8, np.array([40, 40], dtype=np.int32)
    eng = DecodeEngine(30, 1, 2, max_blocks=blocks, max_pos=256, kv=kv)
    eng.slab.zero_()
    sched = pkv.pkv_sched_create(eng.pool, 1, blocks, 128, 4, pkv.PKV_SCHED_CONTINUOUS)
    for rid in (1, 2):
        pkv.pkv_sched_submit(sched, rid, 40, 9)
    _, _, rows = pkv.pkv_sched_admit(sched, 4, 1, blocks)
    own = pkv.pkv_pool_alloc(eng.pool, 3)
    mixed = rows.reshape(1, 2, blocks).copy()
    mixed[0, 0, :3] = own                        # one row the caller's, one a request's
    acc = torch.rand((2, lh.HKV, blocks * lh.PS), device="cuda")
    for bt in (rows.reshape(1, 2, blocks), mixed):
        eng.set_tables(bt)
        before = acc.clone()
        free = pkv.pkv_pool_info(eng.pool)["num_free"]
        with pytest.raises(pkv.PkvError) as e:
            eng.evict(0, lens, acc, 20, 4, 1)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
        assert pkv.pkv_pool_info(eng.pool)["num_free"] == free and np.array_equal(eng.bt_host, bt)
        assert torch.equal(eng.bt.cpu(), torch.from_numpy(bt)) and torch.equal(acc, before)
    # a page that is nobody's
    pkv.pkv_pool_free(eng.pool, own)
    with pytest.raises(pkv.PkvError) as e:
        eng.evict(0, lens, acc, 20, 4, 1)
    assert e.value.status == pkv.PKV_ERR_DOUBLE_FREE or e.value.status == pkv.PKV_ERR_INVALID_ARG
    pkv.pkv_sched_destroy(sched)
    assert pkv.pkv_pool_info(eng.pool)["num_free"] == 30
    # the caller's own: as ever
    eng.build_tables(lens)
    assert eng.evict(0, lens, acc, 20, 4, 1).tolist() == [20, 20]
    assert pkv.pkv_pool_info(eng.pool)["num_free"] == 30 - 4
    assert eng.check_errors() == (pkv.PKV_OK, 0)
    eng.close()
