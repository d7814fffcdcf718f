"""CPU checks of the engine's own bookkeeping for long contexts: an engine without a device, CUDA's
streams stood in for."""
import contextlib
import gc
import weakref

import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from paged_kv_decode_12_gb300.engine import DecodeEngine


@pytest.fixture
def bare(monkeypatch):
    """An engine with none of its buffers, on the CPU."""
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    eng = DecodeEngine.__new__(DecodeEngine)
    eng.device, eng.pool, eng._extra_ws = torch.device("cpu"), None, {}
    return eng


def test_outgrown_workspaces_stay_for_the_graphs_that_hold_them(bare):
    """A captured graph keeps a workspace's address only: the memory must not go to anybody else."""
    made = []
    for nbytes in (100, 5000, 300, 70000):
        ws = bare._workspace("shared", nbytes, None)
        assert ws.numel() >= nbytes and not ws.any()
        made.append((ws.data_ptr(), weakref.ref(ws)))
        del ws
    gc.collect()
    assert [r() is not None and r().data_ptr() == p for p, r in made] == [True] * 4
    # the largest serves what is smaller, and the kinds of call do not share
    assert bare._workspace("shared", 6000, None).data_ptr() == made[-1][0]
    assert bare._workspace("scored", 6000, None).data_ptr() not in [p for p, _ in made]


def test_workspaces_that_grow_a_little_at_a_time_do_not_pile_up(bare):
    for nbytes in range(1000, 100000, 500):
        bare._workspace("shared", nbytes, None)
    assert sum(t.numel() for kept in bare._extra_ws.values() for t in kept) <= 5 * 100000


def test_new_tables_go_where_the_old_ones_were(bare):
    """Captured graphs hold the device tables' address."""
    bare.layers, bare.batch, bare.max_blocks, bare.bt, bare.bt_host = 2, 3, 4, None, None
    first = np.arange(24, dtype=np.int32).reshape(2, 3, 4)
    bare.set_tables(first)
    at = bare.bt.data_ptr()
    second = first[::-1] + 100
    bare.set_tables(second)
    assert bare.bt.data_ptr() == at and np.array_equal(bare.bt.numpy(), second)
    assert np.array_equal(bare.bt_host, second) and bare.bt_host.flags.c_contiguous
    # the caller's array is neither the device's nor changed with it
    own = second.copy()
    bare.set_tables(own)
    own[:] = -5
    assert np.array_equal(bare.bt.numpy(), second)


def test_workspace_of_a_windowed_engine(bare):
    """What the window's calls need for any rows of the batch: not a whole table's, and not nothing where the
    library chooses the units (smaller batches are cut finer)."""
    need = pkv.pkv_decode_window_workspace_bytes
    bare.batch, bare.max_blocks, bare.window, bare.sinks = 256, 2048, 4096, 16
    for ppc in (1, 16, 128):
        bare.pages_per_chunk = ppc
        assert bare._attention_bytes() == need(256, 2048, 4096, 16, ppc) < pkv.pkv_decode_workspace_bytes(256, 2048, ppc)
    bare.pages_per_chunk = 0
    assert bare._attention_bytes() >= max(need(b, 2048, 4096, 16, 0) for b in (1, 2, 3, 5, 8, 64, 100, 256)) > 0
    bare.batch, bare.max_blocks, bare.window, bare.sinks = 64, 63, 1000, 5
    assert bare._attention_bytes() >= max(need(b, 63, 1000, 5, 0) for b in range(1, 65)) > need(64, 63, 1000, 5, 0)
    bare.window = bare.sinks = 0
    bare.pages_per_chunk = 20
    assert bare._attention_bytes() == pkv.pkv_decode_workspace_bytes(64, 63, 20)


def test_shared_refuses_groups_that_it_would_read_past(bare, monkeypatch):
    """The bounds of n groups are n + 1 numbers; both arrays are read as int32 in a row."""
    bare.batch, bare.max_blocks, bare.pages_per_chunk, bare.bt = 4, 8, 4, torch.zeros((1, 4, 8), dtype=torch.int32)
    bare.scale, bare.err, bare.step_options = 0.125, None, 0
    called = []
    monkeypatch.setattr(pkv, "pkv_decode_shared", lambda *a: called.append(a))

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32)

    def call(starts, prefix):
        bare.attention_shared(0, None, None, starts, prefix, 2, None)

    for starts, prefix in ((i32(0, 4), i32(1, 1)), (i32(0, 2, 3, 4), i32(1, 1)), (i32(0), i32(1)), (i32(0, 4), i32()),
                           (torch.tensor([0, 2, 4]), i32(1, 1)), (i32(0, 2, 4), torch.tensor([1, 1])),
                           (i32(0, 9, 2, 9, 4)[::2], i32(1, 1)), (i32(0, 2, 4), i32(1, 9, 1)[::2]),
                           (i32(0, 2, 4).to("meta"), i32(1, 1)), (i32(0, 2, 4), i32(1, 1).to("meta"))):
        with pytest.raises(ValueError):
            call(starts, prefix)
    assert not called
    call(i32(0, 2, 4), i32(1, 1))
    assert len(called) == 1


def test_weights_on_another_device_are_refused(bare):
    bare.batch = 2
    good = torch.zeros(2, 8, 32)
    assert bare._acc_stride(good, good) == 32
    for bad in (good.to("meta"), good.double(), good[:, :, ::2], good[:1], good[0]):
        with pytest.raises(ValueError):
            bare._acc_stride(good, bad)


def test_evictions_refuse_rows_that_lack_pages(bare):
    """Rows behind a shared prefix may have no entries for it, and rows of a window none for what has slid out: an
    eviction would find no rows there, and give back the pages that hold the rest."""
    bare.pool = pkv.pkv_pool_create(0x7F0000000000, 20 * pkv.PKV_PAGE_BYTES)
    bare.layers, bare.batch, bare.max_blocks, bare.bt, bare.err = 1, 2, 4, None, None
    own = pkv.pkv_pool_alloc(bare.pool, 6)
    whole = np.full((1, 2, 4), -1, dtype=np.int32)
    whole[0, 0, :3], whole[0, 1, :3] = own[:3], own[3:]
    acc = torch.zeros(2, 8, 64)
    for hole, lens in (((0, 1, 0), [48, 48]), ((0, 0, 2), [33, 1]), ((0, 1, 1), [16, 17])):
        bt = whole.copy()
        bt[hole] = -1
        bare.set_tables(bt)
        with pytest.raises(ValueError, match="pages"):
            bare.evict(0, np.array(lens, np.int32), acc, 20, 4, 1)
        assert pkv.pkv_pool_info(bare.pool)["num_free"] == 14 and np.array_equal(bare.bt_host, bt)
    pkv.pkv_pool_destroy(bare.pool)
    bare.pool = None
