"""Steps of chunks as they are used: tables, append and attention one after another through the engine, in
captured graphs, beside decode steps and evictions; waits that give up; pages past 32 bits."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from paged_kv_decode_12_gb300.engine import DecodeEngine
from tests import chunk_helpers as ch
from tests import long_helpers as lh
from tests import test_gpu_chunk_append as ta
from tests import test_gpu_long as tl
from tests.test_gpu_long_engine import bf16_dev, rows_of

pytestmark = pytest.mark.gpu

PS, HKV, HQ, D = lh.PS, lh.HKV, lh.HQ, lh.D
KV = ["bf16", "fp8"]
native = tl.native


def i32(*a):
    return lh.dev(np.array(a, np.int32))


class Steps:
    """An engine that starts without a token, and the rows its pages should hold."""

    def __init__(self, kv, B, layers=2, pages=400, blocks=40, T=200, norm=False, seed=0, **kw):
        self.rng = np.random.default_rng(seed)
        self.kv, self.B, self.layers, self.T = kv, B, layers, T
        self.eng = DecodeEngine(pages + 50, layers, B, max_blocks=blocks, pages_per_chunk=4, max_pos=2048, kv=kv, **kw)
        self.eng.set_tables(np.full((layers, B, blocks), -1, np.int32))
        self.pages, self.used = self.eng.take_pages(pages), i32(0)
        self.lens_dev, self.new_dev = i32(*[0] * B), i32(*[0] * B)
        self.starts, self.pos = i32(*[0] * (B + 1)), i32(*[0] * T)
        self.slots = torch.zeros((layers, T), dtype=torch.int64, device="cuda")
        self.qw, self.kw = (bf16_dev(self.rng, (D,)) for _ in range(2)) if norm else (None, None)
        self.q = torch.zeros((layers, T, HQ, D), dtype=torch.bfloat16, device="cuda")
        self.kvs = torch.zeros((layers, T, 2, HKV, D), dtype=torch.bfloat16, device="cuda")
        self.q_out, self.out = torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.cached = np.zeros(B, int)

    def launch(self, stream=None):
        e = self.eng
        e.chunk_tables(self.lens_dev, self.new_dev, self.pages, self.used, self.starts, self.pos, self.slots, stream=stream)
        for l in range(self.layers):
            e.chunk_append(self.kvs[l, :, 0], self.kvs[l, :, 1], self.q[l], self.slots[l], self.pos, self.q_out[l], self.qw,
                           self.kw, stream=stream)
            e.chunk_attention(l, self.q_out[l], self.lens_dev, self.starts, self.out[l], stream=stream)

    def fill(self, new):
        self.new = np.array(new)
        self.new_dev.copy_(lh.dev(self.new.astype(np.int32)))
        self.q.copy_(bf16_dev(self.rng, self.q.shape))
        self.kvs.copy_(bf16_dev(self.rng, self.kvs.shape))
        self.out.fill_(ch.SENTINEL)

    def check(self):
        """The step's rows in the pages and its outputs, from what the pages hold."""
        torch.cuda.synchronize()
        e, new, cached = self.eng, self.new, self.cached
        assert e.check_errors() == (pkv.PKV_OK, 0)
        e.read_tables()
        n = int(new.sum())
        assert self.lens_dev.tolist() == (cached + new).tolist()
        assert self.starts.tolist() == [0] + np.cumsum(new).tolist()
        pos = np.concatenate([np.arange(c, c + m) for c, m in zip(cached, new)] + [np.zeros(self.T - n, int)])
        assert self.pos.tolist() == pos.tolist()
        pages = e.bt_host[e.bt_host >= 0]
        assert np.unique(pages).size == pages.size == int(self.used)
        axes = np.stack([pos[:n]] * 3)
        for l in range(self.layers):
            ta.rounded_once(self.q_out[l, :n].cpu(), ta.formula(self.q[l, :n].cpu(), self.qw_host(self.qw), 1e-5, axes, None), "q",
                            2.0 ** -20)
            want_k = ta.formula(self.kvs[l, :n, 0].cpu(), self.qw_host(self.kw), 1e-5, axes, None)
            qf, out, at = lh.bf16_values(self.q_out[l]), lh.bf16_values(self.out[l]), 0
            assert (out[n:] == ch.SENTINEL).all()
            for b in range(self.B):
                if not new[b]:
                    continue
                K, V = rows_of(e, self.kv, l, b, range(cached[b] + new[b]))
                mine = want_k[at:at + new[b]].transpose(1, 0, 2)
                v = lh.bf16_values(self.kvs[l, at:at + new[b], 1]).transpose(1, 0, 2)
                for got, want in ((K[:, cached[b]:], mine), (V[:, cached[b]:], v)):
                    # BF16: half a step (2^-8); FP8: another 2^-4, or half the smallest step 2^-9 / 448 of the row's largest
                    off = 2.0 ** -8 * np.abs(want) * 1.01 + 2.0 ** -30
                    if self.kv == "fp8":
                        off = off + 2.0 ** -4 * 1.01 * np.abs(want) + 2.0 ** -10 / 448 * 1.01 * np.abs(want).max(-1, keepdims=True)
                    assert (np.abs(got - want) <= off).all(), (l, b)
                for i in range(new[b]):
                    tokens = ch.seen(cached[b] + i, e.window, e.sinks)
                    o, off = ch.attend(qf[at + i], K[:, tokens], V[:, tokens], self.kv)
                    assert (np.abs(out[at + i] - o) <= off).all(), (l, b, i)
                at += new[b]
        self.cached = cached + new

    @staticmethod
    def qw_host(w):
        return None if w is None else w.cpu()


PLAN = [[37, 1, 0, 64, 5], [1, 33, 16, 1, 0], [1, 1, 1, 1, 1], [0, 0, 90, 3, 0], [0, 0, 0, 0, 0], [15, 1, 1, 40, 17]]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("norm,window,sinks", [(True, 0, 0), (False, 0, 0), (True, 30, 3)])
def test_steps_one_after_another(kv, norm, window, sinks):
    s = Steps(kv, 5, norm=norm, window=window, sinks=sinks)
    for new in PLAN:
        s.fill(new)
        s.launch()
        s.check()
    s.eng.close()


@pytest.mark.parametrize("kv", KV)
def test_steps_replayed_from_one_graph_with_many_sequences(kv):
    """20 sequences: single tokens go beside the chunks; the arrays are as large as the largest step."""
    s = Steps(kv, 20, layers=1, norm=True, pages=800, T=260)
    s.fill([0] * 20)
    s.launch()                                    # (makes the workspaces)
    s.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.launch()
    torch.cuda.synchronize()
    for new in ([13] * 20, [1] * 20, [1, 0] * 9 + [100, 34], [70] + [1] * 19, [0, 2] * 10):
        s.fill(new)
        g.replay()
        s.check()
    s.eng.close()


def test_two_graphs_share_the_engine_s_workspaces():
    """Replayed one after the other, in any order, without a wait between."""
    s = Steps("bf16", 20, layers=1, pages=800, T=260)
    s.fill([11] * 20)
    s.launch()
    s.check()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.eng.chunk_attention(0, s.q_out[0], s.lens_dev, s.starts, s.out[0])
        graphs.append(g)
    want = s.out.clone()
    for k in (0, 1, 1, 0, 0, 1):
        s.out.fill_(3.0)
        graphs[k].replay()
        graphs[1 - k].replay()
        torch.cuda.synchronize()
        n = int(s.starts[-1])
        assert torch.equal(s.out[0, :n], want[0, :n]) and (s.out[0, n:] == 3).all()
    s.eng.close()


def test_two_engines_on_two_streams_at_once():
    a, b = (Steps("bf16", 6, layers=2, pages=300, T=180, seed=i) for i in range(2))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for new in ([30] * 6, [1, 50, 1, 1, 0, 100], [1] * 6):
        for s in (a, b):
            s.fill(new)
        torch.cuda.synchronize()
        for s, stream in zip((a, b), streams):
            s.launch(stream)
        for s in (a, b):
            s.check()
    for s in (a, b):
        s.eng.close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("fused", [True, False])
def test_chunks_then_decode_steps_then_an_eviction(kv, fused):
    s = Steps(kv, 4, layers=2, pages=200, T=120, fused=fused)
    e, rng = s.eng, s.rng
    s.fill([50, 17, 1, 33])
    s.launch()
    s.check()
    # a decode step behind it: room from the tables call, the step's own append and attention
    s.fill([1, 1, 1, 1])
    e.chunk_tables(s.lens_dev, s.new_dev, s.pages, s.used, s.starts, s.pos, s.slots)
    q, k, v = (bf16_dev(rng, (2, 4, h, D)) for h in (HQ, HKV, HKV))
    out = torch.empty_like(q)
    given = q.clone()
    e.step(q, k, v, s.pos[:4].contiguous(), s.lens_dev, out)
    torch.cuda.synchronize()
    assert e.check_errors() == (pkv.PKV_OK, 0)
    e.read_tables()
    s.cached = s.cached + 1
    for l in range(2):
        for b in range(4):
            K, V = rows_of(e, kv, l, b, range(s.cached[b]))
            turned = lh.rotated(lh.bf16_values(given[l, b]), int(s.cached[b]) - 1)
            qf = torch.from_numpy(turned).to(torch.bfloat16).double().numpy()
            o, off, p, _ = lh.attend(qf, K, V, kv)
            # a query value may be rounded the other way (2^-7 of it): scores off by that of the products' sum
            ds = lh.SCALE * 2.0 ** -8 * np.abs(np.einsum("hd,hnd->hn", np.abs(qf), np.abs(np.repeat(K, 4, 0)))).max(-1)
            off = off + np.expm1(2 * 2 * ds)[:, None] * np.einsum("hn,hnd->hd", p, np.abs(np.repeat(V, 4, 0)))
            assert (np.abs(lh.bf16_values(out[l, b]) - o) <= off).all(), (l, b)
    # caches cut, from the tables as they are on the device
    free = pkv.pkv_pool_info(e.pool)["num_free"]
    acc = torch.from_numpy(rng.random((2, 4, HKV, 40 * PS)).astype(np.float32)).cuda()
    lens = s.cached.astype(np.int32)
    weights = acc.cpu().numpy()
    for l in range(2):
        before = [rows_of(e, kv, l, b, range(lens[b])) for b in range(4)]
        after = e.evict(l, lens, acc[l], 20, 6, 2)
        assert after.tolist() == np.minimum(lens, 20).tolist()
        for b in range(4):
            K, V = rows_of(e, kv, l, b, range(after[b]))
            for g in range(HKV):
                ids = tl.plain_evict(weights[l, b, g], int(lens[b]), 20, 6, 2)
                assert np.array_equal(K[g], before[b][0][g, ids]) and np.array_equal(V[g], before[b][1][g, ids])
    held = 2 * int((-(-np.minimum(lens, 20) // PS)).sum())
    assert pkv.pkv_pool_info(e.pool)["num_free"] == free + int(s.used) - held
    # and more chunks behind the cut caches (positions are places again)
    s.cached = np.minimum(lens, 20)
    s.lens_dev.copy_(lh.dev(s.cached.astype(np.int32)))
    s.fill([3, 40, 0, 1])
    s.launch()
    torch.cuda.synchronize()
    assert e.check_errors() == (pkv.PKV_OK, 0)
    n = int(s.new.sum())
    e.read_tables()
    for l in range(2):
        qf, got, at = lh.bf16_values(s.q_out[l]), lh.bf16_values(s.out[l]), 0
        for b in range(4):
            K, V = rows_of(e, kv, l, b, range(s.cached[b] + s.new[b]))
            for i in range(s.new[b]):
                o, off = ch.attend(qf[at], K[:, :s.cached[b] + i + 1], V[:, :s.cached[b] + i + 1], kv)
                assert (np.abs(got[at] - o) <= off).all(), (l, b, i)
                at += 1
        assert at == n
    e.close()


def test_a_list_that_runs_out_is_replaced():
    s = Steps("bf16", 3, layers=2, pages=8, T=64)
    s.fill([20, 16, 16])                          # 2 * 4 pages
    s.launch()
    s.check()
    s.fill([1, 1, 20])
    before = [x.clone() for x in (s.eng.bt, s.lens_dev, s.eng.slab)]
    s.launch()
    assert s.eng.check_errors()[1] == pkv.PKV_DEVERR_PAGES
    for x, y in zip(before, (s.eng.bt, s.lens_dev, s.eng.slab)):
        assert torch.equal(x, y)
    assert (s.out == ch.SENTINEL).all()           # no sequence brought anything
    s.eng.err.zero_()
    s.pages.copy_(s.eng.take_pages(8))
    s.used.zero_()
    s.launch()
    used = int(s.used)
    s.used += 8                                   # (all that are taken, for the check)
    s.check()
    assert used == 2 * 3
    s.eng.close()


def test_the_engine_s_refusals():
    s = Steps("bf16", 3, layers=2, pages=8, T=64)
    e = s.eng
    for change in (dict(lens_dev=s.lens_dev.long()), dict(new_dev=s.new_dev[:2]), dict(used=i32(0, 0)), dict(starts=s.starts[:3]),
                   dict(slots=s.slots[:1]), dict(slots=s.slots.int()), dict(pos=s.pos[::2]), dict(pages=s.pages.cpu())):
        a = dict(lens_dev=s.lens_dev, new_dev=s.new_dev, pages=s.pages, used=s.used, starts=s.starts, pos=s.pos, slots=s.slots)
        with pytest.raises(ValueError):
            e.chunk_tables(*dict(a, **change).values())
    k, v = s.kvs[0, :, 0], s.kvs[0, :, 1]
    for change in (dict(k=k.float()), dict(v=v[:5]), dict(q=s.q[0].transpose(1, 2)), dict(slots=s.slots[0].int()),
                   dict(pos=s.pos.long()), dict(pos=torch.zeros((2, 64), dtype=torch.int32, device="cuda"), axis_pairs=(8, 12, 12)),
                   dict(q_out=torch.zeros((64, HQ + 1, D), dtype=torch.bfloat16, device="cuda")[:, :HQ]),
                   dict(q_norm=bf16_dev(s.rng, (32,))), dict(k_norm=torch.ones(64, device="cuda"))):
        a = dict(k=k, v=v, q=s.q[0], slots=s.slots[0], pos=s.pos)
        with pytest.raises(ValueError):
            e.chunk_append(**dict(a, **change))
    with pytest.raises(pkv.PkvError):             # one norm without the other
        e.chunk_append(k, v, s.q[0], s.slots[0], s.pos, k_norm=bf16_dev(s.rng, (D,)))
    for change in (dict(q=s.q[0].float()), dict(q=s.q[0, :, :, :32]), dict(out=s.out[0, :3]), dict(starts=s.starts[:-1]),
                   dict(seq_lens_dev=s.lens_dev.cpu())):
        a = dict(q=s.q[0], seq_lens_dev=s.lens_dev, starts=s.starts, out=s.out[0])
        with pytest.raises(ValueError):
            e.chunk_attention(0, **dict(a, **change))
    torch.cuda.synchronize()
    assert e.check_errors() == (pkv.PKV_OK, 0) and not s.slots.any() and not s.lens_dev.any()
    e.close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("sizes", [[(900, 70), (0, 200), (300, 33)], [(700, 1)], [(500, 1)] * 10 + [(200, 150)] * 9,
                                   [(6000, 64)]])
def test_waits_that_give_up_end(kv, sizes):
    b = ch.Batch(kv, sizes, seed=21).upload().call()
    assert b.flag() == 0
    want = b.out.clone()
    for _ in range(2):
        b.call(options=pkv.PKV_STEP_TEST_EXPIRE_WAIT)
        assert b.flag() == pkv.PKV_DEVERR_TIMEOUT
        b.err.zero_()
        b.out.fill_(ch.SENTINEL)
        b.call()
        assert b.flag() == 0 and torch.equal(b.out, want)
    b.close()


@pytest.mark.parametrize("kv", KV)
def test_pages_past_32_bits(kv):
    """Pages whose bytes lie past 4 GiB of the slab: appended to and read."""
    page = pkv.PKV_PAGE_BYTES if kv == "bf16" else pkv.PKV_PAGE_BYTES_FP8
    pages = (5 << 30) // page
    b = ch.Batch(kv, [(100, 40), (37, 1)], seed=31).upload()
    slab = torch.zeros(pages * page, dtype=torch.uint8, device="cuda")
    base = pages - b.cache.pages
    slab[base * page:] = b.cache.slab
    make = pkv.pkv_pool_create if kv == "bf16" else pkv.pkv_pool_create_fp8
    pool = make(slab, slab.numel())
    b.dev["bt"] = torch.where(b.dev["bt"] >= 0, b.dev["bt"] + base, b.dev["bt"])
    small = b.cache.pool
    b.cache.pool = pool
    b.call()
    assert b.flag() == 0
    b.check()
    b.cache.pool = small
    # a token's row to the last page
    rng = np.random.default_rng(32)
    k, v = bf16_dev(rng, (1, HKV, D)), bf16_dev(rng, (1, HKV, D))
    last = np.full(1, pages * PS - 1, np.int64)
    rope = pkv.rope_table(64, "cuda")
    for p, slots in ((pool, last), (small, last - base * PS)):
        pkv.pkv_chunk_append(p, k, 512, v, 512, None, 0, None, None, None, 0.0, lh.dev(slots), i32(5), 0, None, 1, rope, 64, b.err)
    assert b.flag() == 0 and torch.equal(slab[base * page:], b.cache.slab)
    assert not slab[:base * page].any()
    pkv.pkv_pool_destroy(pool)
    b.close()
