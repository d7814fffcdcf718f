"""Block tables, positions and slots made on the GPU, against the rules written out in numpy.  All
values are whole numbers and have to be equal."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import long_helpers as lh

pytestmark = pytest.mark.gpu

PS = lh.PS


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


def rules(lens, new, bt, max_blocks, pages, used, max_tokens, num_pages):
    """(bt, used, starts, lens, pos, slots, flag) after the call."""
    lens, new = np.asarray(lens, np.int64), np.asarray(new, np.int64)
    layers, B, _ = bt.shape
    ok = (lens >= 0) & (new >= 0) & (lens + new <= PS * max_blocks)
    flag = 0 if ok.all() else pkv.PKV_DEVERR_LENGTH
    n = np.where(ok, new, 0)
    add = np.where(ok, -(-(lens + n) // PS) - -(-lens // PS), 0)
    if n.sum() > max_tokens:
        flag |= pkv.PKV_DEVERR_LENGTH
    short = used < 0 or used + layers * add.sum() > len(pages)
    if short:
        flag |= pkv.PKV_DEVERR_PAGES
    if short or n.sum() > max_tokens:
        n, add = np.zeros_like(n), np.zeros_like(add)
    bt = bt.copy()
    at = used
    for l in range(layers):
        for b in range(B):
            had = -(-lens[b] // PS) if ok[b] else 0
            for i in range(add[b]):
                good = 0 <= pages[at] < num_pages
                bt[l, b, had + i] = pages[at] if good else -1
                flag |= 0 if good else pkv.PKV_DEVERR_PAGE_RANGE
                at += 1
    starts = np.concatenate([[0], np.cumsum(n)])
    pos = np.zeros(max_tokens, np.int64)
    slots = np.full((layers, max_tokens), -1, np.int64)
    for b in range(B):
        for i in range(n[b]):
            t, p = starts[b] + i, lens[b] + i
            pos[t] = p
            for l in range(layers):
                page = int(bt[l, b, p // PS])
                if 0 <= page < num_pages:
                    slots[l, t] = page * PS + p % PS
                else:
                    flag |= pkv.PKV_DEVERR_PAGE_RANGE
    return bt, at, starts, lens + n, pos, slots, flag


def pool_of(num_pages):
    # (the call only asks the pool how many pages it has)
    slab = torch.empty(num_pages * pkv.PKV_PAGE_BYTES_FP8, dtype=torch.uint8, device="cuda")
    return slab, pkv.pkv_pool_create_fp8(slab, slab.numel())


class Call:
    def __init__(self, lens, new, layers, blocks, pages, used, max_tokens, num_pages, bt=None, inplace=False):
        self.B, self.layers, self.blocks, self.max_tokens, self.num_pages = len(lens), layers, blocks, max_tokens, num_pages
        i32 = dict(dtype=torch.int32, device="cuda")
        self.slab, self.pool = pool_of(num_pages)
        self.lens, self.new = (torch.tensor(np.asarray(x), **i32) for x in (lens, new))
        self.bt = torch.tensor(bt, **i32) if bt is not None else torch.full((layers, self.B, blocks), -1, **i32)
        self.pages, self.used = torch.tensor(np.asarray(pages), **i32), torch.tensor([used], **i32)
        self.lens_out = self.lens if inplace else torch.full_like(self.lens, -9)
        self.used_out = self.used if inplace else torch.full_like(self.used, -9)
        self.starts = torch.full((self.B + 1,), -9, **i32)
        self.pos = torch.full((max_tokens,), -9, **i32)
        self.slots = torch.full((layers, max_tokens), -9, dtype=torch.int64, device="cuda")
        self.nbytes = pkv.pkv_chunk_tables_workspace_bytes(self.B)
        self.ws = torch.zeros(self.nbytes, dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, **i32)

    def run(self, stream=None):
        pkv.pkv_chunk_tables(self.pool, self.lens, self.new, self.B, self.bt, self.blocks, self.layers, self.pages,
                             self.pages.numel(), self.used, self.used_out, self.max_tokens, self.starts, self.lens_out,
                             self.pos, self.slots, self.ws, self.nbytes, self.err, stream)
        return self

    def state(self):
        return tuple(x.cpu().numpy() for x in (self.bt, self.used_out, self.starts, self.lens_out, self.pos, self.slots))

    def check(self, want):
        for name, got, w in zip(("bt", "used", "starts", "lens", "pos", "slots"), self.state(), want):
            assert np.array_equal(got.reshape(-1), np.asarray(w).reshape(-1)), name
        assert int(self.err) == want[-1]
        assert not self.ws.any()

    def close(self):
        pkv.pkv_pool_destroy(self.pool)


def held_tables(rng, lens, layers, blocks, ids):
    bt = np.full((layers, len(lens), blocks), -1, np.int32)
    at = 0
    for l in range(layers):
        for b, L in enumerate(lens):
            n = -(-max(int(L), 0) // PS)
            if n <= blocks:
                bt[l, b, :n] = ids[at:at + n]
                at += n
    return bt, at


def make(rng, lens, new, layers, blocks, used=0, extra=0, pad=0, **kw):
    lens, new = np.asarray(lens), np.asarray(new)
    held = layers * int((-(-np.maximum(lens, 0) // PS)).sum())
    need = layers * int((-(-np.maximum(lens + np.maximum(new, 0), 0) // PS)).sum())
    num = held + need + used + extra + 3
    ids = rng.permutation(num).astype(np.int32)
    bt, at = held_tables(rng, lens, layers, blocks, ids)
    pages = ids[at:at + used + (need - held if need > held else 0) + extra]
    T = max(1, int(np.maximum(new, 0).sum()) + pad)
    call = Call(lens, new, layers, blocks, pages, used, T, num, bt, **kw)
    return call, rules(lens, new, bt, blocks, pages, used, T, num)


SIZES = [
    ([0], [1], 1, 0), ([0], [0], 1, 3), ([15], [1], 3, 0), ([16], [1], 3, 0), ([15], [2], 16, 5), ([0, 0, 0], [16, 0, 17], 2, 0),
    ([1, 16, 31, 32, 33], [1, 1, 1, 1, 1], 16, 0), ([100, 0, 48], [0, 0, 0], 4, 7), ([700], [1], 16, 0),
    ([5, 300, 0, 17, 2000], [40, 1, 333, 0, 48], 16, 100), ([0], [2048], 5, 1),
]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_sizes(case, inplace):
    lens, new, layers, pad = SIZES[case]
    call, want = make(np.random.default_rng(case), lens, new, layers, 131, used=case, extra=2, pad=pad, inplace=inplace)
    call.run().check(want)
    call.close()


@pytest.mark.parametrize("B,layers,longest,chunk", [(64, 16, 500, 60), (513, 3, 90, 40), (1025, 1, 40, 20), (4096, 2, 40, 5),
                                                    (200, 33, 70, 30)])
def test_random_batches(B, layers, longest, chunk):
    rng = np.random.default_rng(B)
    lens, new = rng.integers(0, longest, B), rng.integers(0, chunk, B) * (rng.random(B) < 0.7)
    call, want = make(rng, lens, new, layers, 40, used=11, extra=1, pad=int(rng.integers(0, 50)))
    call.run().check(want)
    call.close()


def test_rows_that_are_refused_bring_nothing():
    rng = np.random.default_rng(3)
    lens, new = [20, -1, 30, 16 * 9, 5], [3, 4, -2, 1, 20]
    call, want = make(rng, lens, new, 2, 9, extra=3)
    assert want[-1] == pkv.PKV_DEVERR_LENGTH
    call.run().check(want)
    assert call.lens_out.tolist() == [23, -1, 30, 144, 25]
    call.close()


@pytest.mark.parametrize("what", ["pages", "tokens", "used", "nothing listed"])
def test_all_or_nothing(what):
    rng = np.random.default_rng(4)
    call, _ = make(rng, [20, 0, 30], [30, 5, 16], 2, 9)
    if what == "pages":
        call.pages = call.pages[:-1].contiguous()
    elif what == "used":
        call.used.fill_(-1)
    elif what == "nothing listed":
        call.pages = call.pages[:0].contiguous()
    else:
        call.max_tokens -= 1
        call.pos, call.slots = call.pos[:-1].contiguous(), call.slots[:, :-1].contiguous()
    before = call.bt.clone()
    call.run()
    assert int(call.err) == (pkv.PKV_DEVERR_LENGTH if what == "tokens" else pkv.PKV_DEVERR_PAGES)
    assert torch.equal(call.bt, before) and torch.equal(call.lens_out, call.lens) and torch.equal(call.used_out, call.used)
    assert not call.starts.any() and not call.pos.any() and (call.slots == -1).all()
    call.close()


def test_bad_page_ids():
    rng = np.random.default_rng(5)
    call, _ = make(rng, [20, 7, 32], [30, 5, 16], 2, 9)
    call.bt[1, 1, 0] = call.num_pages           # the partial page of a row in one layer
    call.pages[1] = -4                          # a new page of row 0 in layer 0
    want = rules([20, 7, 32], [30, 5, 16], call.bt.cpu().numpy(), 9, call.pages.cpu().numpy(), 0, call.max_tokens, call.num_pages)
    assert want[-1] == pkv.PKV_DEVERR_PAGE_RANGE
    call.run().check(want)
    call.close()


def test_steps_replayed_in_place_from_a_graph():
    """A captured call that writes its own lengths and count: every replay is the next step."""
    rng = np.random.default_rng(6)
    lens, new = np.array([3, 0, 40, 15]), np.array([1, 7, 0, 18])
    layers, blocks, num = 3, 30, 400
    ids = rng.permutation(num).astype(np.int32)
    bt, at = held_tables(rng, lens, layers, blocks, ids)
    call = Call(lens, new, layers, blocks, ids[at:], 0, 40, num, bt, inplace=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call.run()
    torch.cuda.synchronize()
    used = 0
    for step in range(6):
        new = rng.integers(0, 12, 4)
        call.new.copy_(torch.tensor(new))
        g.replay()
        torch.cuda.synchronize()
        want = rules(lens, new, bt, blocks, ids[at:], used, 40, num)
        call.check(want)
        bt, used, lens = want[0], want[1], want[3]
    call.close()


def test_slots_past_32_bits():
    """16 * page + place does not fit 32 bits."""
    num = 2 ** 31 // PS + 10
    slab = torch.empty(16, dtype=torch.uint8, device="cuda")
    pool = pkv.pkv_pool_create_fp8(slab, num * pkv.PKV_PAGE_BYTES_FP8)
    call = Call([0, 17], [5, 20], 1, 4, [num - 1, num - 2, num - 3], 0, 25, 16, [[[-1] * 4, [num - 4, num - 5, -1, -1]]])
    pkv.pkv_pool_destroy(call.pool)
    call.pool = pool                            # (its pages are never touched)
    want = rules([0, 17], [5, 20], np.array([[[-1] * 4, [num - 4, num - 5, -1, -1]]]), 4, [num - 1, num - 2, num - 3], 0, 25, num)
    assert want[5].max() > 2 ** 31
    call.run().check(want)
    call.close()
