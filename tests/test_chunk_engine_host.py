"""CPU checks of the engine's bookkeeping for steps of chunks: an engine without a device, whose tables are extended
here as chunk_tables does it."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from paged_kv_decode_12_gb300 import workloads as wl
from tests.test_long_engine_host import bare  # noqa: F401 -- the fixture

PS = wl.PAGE_SIZE
PAGES = 120


@pytest.fixture
def eng(bare, monkeypatch):  # noqa: F811
    bare.pool = pkv.pkv_pool_create(0x7F0000000000, PAGES * pkv.PKV_PAGE_BYTES)
    bare.layers, bare.batch, bare.max_blocks, bare.bt, bare.bt_host, bare.err = 2, 3, 12, None, None, None
    bare.set_tables(np.full((2, 3, 12), -1, np.int32))
    monkeypatch.setattr(pkv, "pkv_evict", lambda *a: None)
    yield bare
    pkv.pkv_pool_destroy(bare.pool)
    bare.pool = None


def free(eng):
    return pkv.pkv_pool_info(eng.pool)["num_free"]


class Chunks:
    """Steps as chunk_tables makes them: pages from a list, behind each sequence's last one."""

    def __init__(self, eng, pages):
        self.eng, self.list, self.used = eng, eng.take_pages(pages).numpy(), 0
        self.lens = np.zeros(eng.batch, np.int32)

    def step(self, new):
        for l in range(self.eng.layers):
            for b in range(self.eng.batch):
                had, need = -(-self.lens[b] // PS), -(-(self.lens[b] + new[b]) // PS)
                for i in range(had, need):
                    self.eng.bt[l, b, i] = int(self.list[self.used])
                    self.used += 1
        self.lens = self.lens + np.array(new, np.int32)
        self.eng._device_tables = True

    def evict(self, keep, room):
        acc = torch.zeros(3, 8, 12 * PS)
        for l in range(self.eng.layers):
            after = self.eng.evict(l, self.lens, acc, keep, 4, 1, room=room)
        self.lens = after

    def held(self):
        """Pages that some sequence's tokens are in."""
        return self.eng.layers * int((-(-self.lens // PS)).sum())


def named(eng):
    ids = eng.bt.numpy()[eng.bt.numpy() >= 0]
    assert np.unique(ids).size == ids.size
    return set(ids.tolist())


@pytest.mark.parametrize("room", [0, 1, 40, 1000])
def test_evictions_with_room_and_chunks_do_not_use_the_pool_up(eng, room):
    c = Chunks(eng, 0)
    for cycle in range(12):
        c.list, c.used = eng.take_pages(24).numpy(), 0
        c.step([20, 1, 30])
        c.step([5, 33, 0])
        pkv.pkv_pool_free(eng.pool, c.list[c.used:])                 # those that are still the list's
        c.evict(32, room)
        extra = sum(x.size for x in eng._room.values())
        assert free(eng) == PAGES - c.held() - extra
        assert len(named(eng)) == c.held() + extra
    # the room's pages in use: a token in each sequence's next page, as an append does it, and chunks behind them
    if room == 40:
        c.lens = c.lens + 20
        c.list, c.used = eng.take_pages(24).numpy(), 0
        c.step([30, 30, 30])
        left = c.list[c.used:]
        table = eng.read_tables()
        assert np.array_equal(table, eng.bt.numpy())
        assert free(eng) == PAGES - left.size - len(named(eng))
        assert len(named(eng)) == c.held()


def test_the_room_goes_back_when_it_is_replaced_and_not_before(eng):
    c = Chunks(eng, 12)
    c.step([16, 16, 16])
    c.evict(16, 32)                                                  # 6 pages more a layer
    room = set(np.concatenate(list(eng._room.values())).tolist())
    assert len(room) == 12 and room <= named(eng)
    list_left = 12 - c.used
    before = free(eng)
    eng.read_tables()
    assert free(eng) == before                                       # still named: nothing goes back
    c.list, c.used = eng.take_pages(10).numpy(), 0
    c.step([3, 0, 20])                                               # 1 and 2 pages in each layer
    before = free(eng)
    eng.read_tables()
    assert free(eng) == before + 6 and len(room & named(eng)) == 6
    before = free(eng)
    eng.read_tables()
    assert free(eng) == before
    assert list_left == 12 - 6


def test_pages_that_the_caller_has_taken_stay_with_the_caller(eng):
    """A caller may give back the pages of a sequence that has ended, its room among them, and get them again."""
    c = Chunks(eng, 12)
    c.step([16, 16, 16])
    c.evict(16, 16)
    row = eng.bt_host[:, 0]
    pkv.pkv_pool_free(eng.pool, np.unique(row[row >= 0]))            # sequence 0 has ended
    c.lens[0] = 0
    c.list, c.used = eng.take_pages(free(eng)).numpy(), 0            # (all there are: those pages are among them)
    mine = set(c.list.tolist())
    assert set(row[row >= 0].tolist()) <= mine
    c.step([40, 1, 1])
    eng.read_tables()
    # sequences 1 and 2 have got a page each a layer, and their room goes back
    assert free(eng) == 4 and not mine & set(pkv.pkv_pool_alloc(eng.pool, 4).tolist())


def test_new_tables_end_the_bookkeeping(eng):
    c = Chunks(eng, 12)
    c.step([16, 16, 16])
    c.evict(16, 16)
    c.list, c.used = eng.take_pages(12).numpy(), 0
    c.step([1, 0, 0])
    before = free(eng)
    eng.set_tables(np.full((2, 3, 12), -1, np.int32))
    assert free(eng) == before + 2 and not eng._room                 # the two that were replaced by then
    before = free(eng)
    eng.read_tables()
    assert free(eng) == before


class Elsewhere(torch.Tensor):
    """A tensor that says it is on some device."""

    @staticmethod
    def on(t, device):
        t = t.as_subclass(Elsewhere)
        t.where = torch.device(device)
        return t

    @property
    def device(self):
        return self.where


def test_arrays_on_another_gpu_are_refused(bare, monkeypatch):  # noqa: F811
    bare.device, here, there = torch.device("cuda:0"), "cuda:0", "cuda:1"
    bare.layers, bare.batch, bare.max_blocks, bare.bt, bare.err = 1, 2, 4, torch.zeros((1, 2, 4), dtype=torch.int32), None
    bare.scale, bare.window, bare.sinks, bare.step_options, bare.rope, bare.max_pos = 0.125, 0, 0, 0, None, 64
    bare.pages_per_chunk = 4
    monkeypatch.setattr(bare, "_workspace", lambda *a: None)
    called = []
    for name in ("pkv_chunk_tables", "pkv_chunk_append", "pkv_chunk_attention", "pkv_decode_shared"):
        monkeypatch.setattr(pkv, name, lambda *a, name=name: called.append(name))

    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32)

    def bf16(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16)

    calls = {
        "chunk_tables": dict(seq_lens_dev=i32(2), new_dev=i32(2), pages_dev=i32(5), used_dev=i32(1), starts=i32(3), pos=i32(7),
                             slots=torch.zeros((1, 7), dtype=torch.int64), seq_lens_out=i32(2), used_out=i32(1)),
        "chunk_append": dict(k=bf16(7, 8, 64), v=bf16(7, 8, 64), q=bf16(7, 32, 64), slots=torch.zeros(7, dtype=torch.int64),
                             pos=i32(7), q_out=bf16(7, 32, 64), q_norm=bf16(64), k_norm=bf16(64)),
        "chunk_attention": dict(q=bf16(7, 32, 64), seq_lens_dev=i32(2), starts=i32(3), out=bf16(7, 32, 64)),
    }
    for call, arrays in calls.items():
        def run(at):
            args = {x: Elsewhere.on(t, at.get(x, here)) for x, t in arrays.items()}
            getattr(bare, call)(**(dict(args, layer=0) if call == "chunk_attention" else args))

        run({})
        assert called.pop() == "pkv_" + call
        for x in arrays:
            with pytest.raises(ValueError):
                run({x: there})
            assert not called, x
    acc = torch.zeros(2, 8, 64)
    assert bare._acc_stride(Elsewhere.on(acc, here)) == 64
    with pytest.raises(ValueError):
        bare._acc_stride(Elsewhere.on(acc, there))
    for starts, prefix in ((there, here), (here, there)):
        with pytest.raises(ValueError):
            bare.attention_shared(0, None, None, Elsewhere.on(i32(2), starts), Elsewhere.on(i32(1), prefix), 2, None)
    assert not called


def test_pages_that_another_eviction_has_taken_stay_with_it(eng):
    """The same where an eviction of another layer gets the pages that the caller has given back."""
    c = Chunks(eng, 12)
    c.step([16, 16, 16])
    eng.read_tables()
    eng._device_tables = False                                       # (as before the first chunk_tables)
    pkv.pkv_pool_alloc(eng.pool, free(eng) - 9)                      # (few pages are left)
    acc = torch.zeros(3, 8, 12 * PS)
    eng.evict(0, c.lens, acc, 16, 4, 1, room=32)
    room = eng._room[0]
    pkv.pkv_pool_free(eng.pool, room)                                # the caller gives layer 0's room back
    keep = eng.bt[0].clone()
    keep[torch.from_numpy(np.isin(eng.bt[0].numpy(), room))] = -1
    eng.bt[0].copy_(keep)
    eng.evict(1, c.lens, acc, 16, 4, 1)                              # takes three of them
    taken = eng.bt_host[1][eng.bt_host[1] >= 0]
    assert np.isin(taken, room).any()
    before = free(eng)
    eng.bt[1].fill_(-1)                                              # (sequences that have ended, pages not given back)
    eng.read_tables()
    assert free(eng) == before
