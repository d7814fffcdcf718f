"""The long-context operators as they are used together: through the engine, in captured graphs, on
two streams at once, and with waits that give up."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from paged_kv_decode_12_gb300.engine import DecodeEngine
from tests import long_helpers as lh
from tests import paged_helpers as ph
from tests import test_gpu_long as tl

pytestmark = pytest.mark.gpu

PS, HKV, HQ, D = lh.PS, lh.HKV, lh.HQ, lh.D
KV = ["bf16", "fp8"]
native = tl.native


def bf16_dev(rng, shape):
    return torch.from_numpy(lh.bf16_bits(rng.standard_normal(shape)).view(np.int16).copy()).view(torch.bfloat16).cuda()


def rows_of(eng, kv, layer, b, tokens):
    """K, V [8][n][64] in FP64 as the engine's pool holds them."""
    c = lh.Cache(kv, 1)
    c.host = eng.slab.cpu().numpy().view(np.uint16 if kv == "bf16" else np.uint8)
    return c.rows(eng.bt_host[layer, b], tokens, c.host)


@pytest.mark.parametrize("kv", KV)
def test_refused_evictions_take_no_pages_and_shared_pages_are_freed_once(kv):
    rng = np.random.default_rng(8)
    lens, blocks = np.array([40, 40, 0], dtype=np.int32), 4
    eng = DecodeEngine(40, 1, 3, max_blocks=blocks, max_pos=256, kv=kv)
    own = eng.build_tables(np.array([40, 33, 1]))
    bt = own.copy()
    spare = int(bt[0, 1, 0])
    bt[0, 1, 0] = bt[0, 0, 0]                    # rows 0 and 1 share their first page
    pkv.pkv_pool_free(eng.pool, [spare])
    eng.set_tables(bt)
    pkv.pkv_prefill_append(eng.pool, *(bf16_dev(rng, (1, 40, HKV, D)) for _ in range(2)), lh.dev(bt[:, 0]), blocks, 1, 0,
                           40, eng.rope, eng.max_pos, eng.err)
    acc = torch.from_numpy(rng.random((3, HKV, blocks * PS)).astype(np.float32)).cuda()
    free = pkv.pkv_pool_info(eng.pool)["num_free"]
    for args, error in (((0, lens, acc, 20, 15, 6), pkv.PkvError),             # sinks + recent > keep
                        ((0, lens, acc, 0, 0, 0), pkv.PkvError),
                        ((0, [40, 65, 0], acc, 20, 4, 1), ValueError),         # a length beyond the table
                        ((0, [40, -1, 0], acc, 20, 4, 1), ValueError),
                        ((0, lens[:2], acc, 20, 4, 1), ValueError),
                        ((0, lens, acc[:, :, ::2], 20, 4, 1), ValueError),
                        ((0, lens, acc.double(), 20, 4, 1), ValueError)):
        with pytest.raises(error):
            eng.evict(*args)
        assert pkv.pkv_pool_info(eng.pool)["num_free"] == free and np.array_equal(eng.bt_host, bt)
    before = rows_of(eng, kv, 0, 0, range(40))
    weights = acc.cpu().numpy()
    assert eng.evict(0, lens, acc, 20, 4, 1).tolist() == [20, 20, 0]
    after = rows_of(eng, kv, 0, 0, range(20))
    for g in range(HKV):
        ids = tl.plain_evict(weights[0, g], 40, 20, 4, 1)
        assert np.array_equal(after[0][g], before[0][g, ids]) and np.array_equal(after[1][g], before[1][g, ids])
    assert (eng.bt_host >= 0).sum() == 4 and np.unique(eng.bt_host[eng.bt_host >= 0]).size == 4
    assert pkv.pkv_pool_info(eng.pool)["num_free"] == 40 - 4
    assert eng.evict(0, [0, 0, 0], acc, 20, 4, 1).tolist() == [0, 0, 0]
    assert pkv.pkv_pool_info(eng.pool)["num_free"] == 40
    assert eng.check_errors() == (pkv.PKV_OK, 0)


def test_first_calls_on_another_stream_and_in_a_capture():
    """A workspace is zeroed on the stream that its call runs on, and never inside a capture."""
    rng = np.random.default_rng(9)
    lens, blocks, B = np.full(4, 200, dtype=np.int32), 16, 4
    eng = DecodeEngine(80, 1, B, max_blocks=blocks, pages_per_chunk=2, max_pos=512)
    eng.build_tables(lens)
    for b in range(B):
        pkv.pkv_prefill_append(eng.pool, *(bf16_dev(rng, (1, 200, HKV, D)) for _ in range(2)),
                               lh.dev(eng.bt_host[:, b]), blocks, 1, 0, 200, eng.rope, eng.max_pos, eng.err)
    q, lens_d = bf16_dev(rng, (B, HQ, D)), lh.dev(lens)
    starts, none = lh.dev(np.array([0, B], dtype=np.int32)), lh.dev(np.zeros(1, dtype=np.int32))
    acc = torch.zeros((B, HKV, blocks * PS), device="cuda")
    want, out, scored = (torch.empty_like(q) for _ in range(3))
    eng.attention(0, q, lens_d, want)
    calls = [lambda st: eng.attention_shared(0, q, lens_d, starts, none, 0, out, stream=st),
             lambda st: eng.attention_scored(0, q, lens_d, acc, acc, scored, stream=st)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin()
        for call in calls:
            with pytest.raises(RuntimeError, match="before it is captured"):
                call(None)
        with pytest.raises(RuntimeError, match="cannot be captured"):
            eng.evict(0, lens, acc, 100, 10)
        q.add_(0)
        graph.capture_end()
    torch.cuda.synchronize()
    # garbage where the workspaces will be, and much work on the current stream
    junk = torch.full((1 << 22,), 7, dtype=torch.int32, device="cuda")
    del junk
    slow = torch.zeros(1 << 26, device="cuda")
    for _ in range(50):
        slow.add_(1)
    for call in calls:
        call(s)
    s.synchronize()
    # the same partials merged in FP32: both round to BF16 values a step (2^-7) apart at most
    for got in (out, scored):
        assert ((got.double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 2.0 ** -30).all()
    # 4 heads' weights add to 1 each, but for the roundings of a sum of 200 (2^-24 each) and of an
    # exponent below 2^4 and its power of two (2^-19)
    sums = acc.cpu().numpy().astype(np.float64).sum(-1)
    assert (np.abs(sums - 4) <= 4 * (200 * 2.0 ** -24 + 2.0 ** -19)).all()
    torch.cuda.synchronize()
    assert eng.check_errors() == (pkv.PKV_OK, 0)


@pytest.mark.parametrize("kv", KV)
def test_scored_steps_evictions_and_more_steps(kv):
    rng = np.random.default_rng(5)
    layers, prompts = 2, np.array([70, 33, 20], dtype=np.int32)
    B, blocks = prompts.size, 8
    eng = DecodeEngine(120, layers, B, max_blocks=blocks, pages_per_chunk=3, max_pos=512, kv=kv)
    eng.build_tables(prompts + 20)
    for b in range(B):
        k, v = (bf16_dev(rng, (layers, prompts[b], HKV, D)) for _ in range(2))
        pkv.pkv_prefill_append(eng.pool, k, v, lh.dev(eng.bt_host[:, b]), blocks, layers, 0, int(prompts[b]), eng.rope,
                               eng.max_pos, eng.err)
    acc = torch.zeros((layers, B, HKV, blocks * PS), device="cuda")
    cached = prompts.copy()                      # tokens in the cache
    at = prompts.copy()                          # the next token's position
    ref = [[rows_of(eng, kv, layer, b, range(prompts[b])) for b in range(B)] for layer in range(layers)]
    want_acc = np.zeros(acc.shape)
    tol_acc = np.zeros(acc.shape)

    def step():
        nonlocal cached, at
        for layer in range(layers):
            q, kn, vn = bf16_dev(rng, (B, HQ, D)), bf16_dev(rng, (B, HKV, D)), bf16_dev(rng, (B, HKV, D))
            out = torch.empty_like(q)
            eng.append(layer, kn, vn, q, lh.dev(at), slots=lh.dev(cached))
            eng.attention_scored(layer, q, lh.dev(cached + 1), acc[layer], acc[layer], out)
            qf = lh.bf16_values(q)               # rotated in place
            for b in range(B):
                new = rows_of(eng, kv, layer, b, [cached[b]])
                want = lh.rotated(lh.bf16_values(kn[b]), at[b])
                step_k = 2.0 ** -7 if kv == "bf16" else 2.0 ** -2
                assert (np.abs(new[0][:, 0] - want) <= step_k * np.abs(want) + 2.0 ** -9 * np.abs(want).max()).all()
                ref[layer][b] = tuple(np.concatenate([x, y], 1) for x, y in zip(ref[layer][b], new))
                K, V = ref[layer][b]
                o, off, p, dp = lh.attend(qf[b], K, V, kv)
                tl.close(out[b], o, off, (layer, b))
                n = K.shape[1]
                w, t = p.reshape(HKV, 4, n).sum(1), dp.reshape(HKV, 4, n).sum(1)
                want_acc[layer, b, :, :n] += w
                tol_acc[layer, b, :, :n] += t + 2.0 ** -20 * w + 2.0 ** -24 * 4 * want_acc[layer, b, :, :n]
        cached, at = cached + 1, at + 1
        got = acc.cpu().numpy().astype(np.float64)
        assert (np.abs(got - want_acc) <= tol_acc).all()

    def cut(keep, recent, sinks):
        nonlocal cached, want_acc, tol_acc
        free = pkv.pkv_pool_info(eng.pool)["num_free"]
        lens = cached.copy()
        held = (eng.bt_host >= 0).sum()
        for layer in range(layers):
            weights = acc[layer].cpu().numpy()
            after = eng.evict(layer, lens, acc[layer], keep, recent, sinks)
            now_acc, now_tol = np.zeros(want_acc.shape[1:]), np.zeros(want_acc.shape[1:])
            for b in range(B):
                K, V = ref[layer][b]
                ids = [tl.plain_evict(weights[b, g], int(lens[b]), keep, recent, sinks) for g in range(HKV)]
                ref[layer][b] = tuple(np.stack([x[g, ids[g]] for g in range(HKV)]) for x in (K, V))
                got = rows_of(eng, kv, layer, b, range(after[b]))
                assert np.array_equal(got[0], ref[layer][b][0]) and np.array_equal(got[1], ref[layer][b][1])
                for g in range(HKV):
                    now_acc[b, g, :after[b]] = want_acc[layer, b, g, ids[g]]
                    now_tol[b, g, :after[b]] = tol_acc[layer, b, g, ids[g]]
            want_acc[layer], tol_acc[layer] = now_acc, now_tol
        assert np.array_equal(after, np.minimum(lens, keep))
        assert pkv.pkv_pool_info(eng.pool)["num_free"] == free + held - (eng.bt_host >= 0).sum()
        cached = after.copy()

    for _ in range(3):
        step()
    cut(41, 10, 2)
    assert cached.tolist() == [41, 36, 23]
    # the tables hold pages for the cut caches only: make room for more tokens
    for layer in range(layers):
        for b in range(B):
            have = int((eng.bt_host[layer, b] >= 0).sum())
            eng.bt_host[layer, b, have:have + 1] = pkv.pkv_pool_alloc(eng.pool, 1)
    eng.set_tables(eng.bt_host)
    for _ in range(4):
        step()
    cut(30, 0, 0)
    assert eng.check_errors() == (pkv.PKV_OK, 0)
    eng.close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("chains", [1, 2])
def test_engine_with_a_window(kv, chains):
    rng = np.random.default_rng(6)
    layers, lens = 2, np.array([150, 40, 97, 16], dtype=np.int32)
    B, window, sinks = lens.size, 30, 5
    made = []
    for fused in (True, False):
        eng = DecodeEngine(80, layers, B, max_blocks=10, pages_per_chunk=2, max_pos=256, kv=kv, fused=fused, chains=chains,
                           window=window, sinks=sinks)
        g = torch.Generator("cuda").manual_seed(3)
        if kv == "bf16":
            eng.pool_view().copy_(torch.randn(eng.pool_view().shape, generator=g, device="cuda"))
        else:
            codes, scales = eng.fp8_views()
            codes.copy_(torch.randint(0, 120, codes.shape, generator=g, device="cuda", dtype=torch.uint8))
            scales.copy_(torch.rand(scales.shape, generator=g, device="cuda") * 0.01)
        eng.build_tables(lens)
        # pages that have slid out of the window are given back
        gone = [(layer, b, j) for layer in range(layers) for b in range(B) for j in range(10)
                if eng.bt_host[layer, b, j] >= 0 and j * PS >= sinks and (j + 1) * PS <= lens[b] - window]
        assert gone
        before = eng.bt_host.copy()
        for i in gone:
            pkv.pkv_pool_free(eng.pool, [eng.bt_host[i]])
            eng.bt_host[i] = -1
        eng.set_tables(eng.bt_host)
        made.append((eng, before))
    q0 = bf16_dev(rng, (layers, B, HQ, D))
    kn, vn = bf16_dev(rng, (layers, B, HKV, D)), bf16_dev(rng, (layers, B, HKV, D))
    outs = []
    for eng, before in made:
        q, out = q0.clone(), torch.empty_like(q0)
        eng.step(q, kn, vn, lh.dev(lens - 1), lh.dev(lens), out)
        assert eng.check_errors() == (pkv.PKV_OK, 0)
        outs.append((q, out, eng.slab.clone()))
        for layer in range(layers):
            for b in range(B):
                t = tl.visible(int(lens[b]), window, sinks)
                K, V = rows_of(eng, kv, layer, b, t)
                want, off, _, _ = lh.attend(lh.bf16_values(q[layer, b]), K, V, kv)
                tl.close(out[layer, b], want, off, (layer, b))
        eng.close()
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_engine_refuses_windows_it_cannot_have():
    for kw in (dict(window=-1), dict(window=4, sinks=-1), dict(sinks=4), dict(window=4, split_merge=True, fused=False)):
        with pytest.raises(ValueError):
            DecodeEngine(8, 1, 1, max_blocks=4, **kw)


@pytest.mark.parametrize("kv", KV)
def test_engine_shared_prefix(kv):
    groups = [(9, [20, 5, 33]), (2, [7, 40])]
    c, bt, view, lens, starts, prefix, rng = tl.shared_case(kv, groups, 31)
    B = lens.size
    eng = DecodeEngine(c.pages, 1, B, max_blocks=bt.shape[1], pages_per_chunk=4, kv=kv)
    eng.slab.copy_(c.slab)
    eng.set_tables(bt[None])
    q, qf = lh.query(rng, B)
    out = torch.empty_like(q)
    for _ in range(2):                            # the workspace is kept and used again
        eng.attention_shared(0, q, lh.dev(lens), lh.dev(starts), lh.dev(prefix), int(prefix.max()), out)
    assert eng.check_errors() == (pkv.PKV_OK, 0)
    for b in range(B):
        K, V = c.rows(view[b], range(int(lens[b])))
        tl.close(out[b], *lh.attend(qf[b], K, V, kv, 2.0 ** -8)[:2])
    eng.close()
    c.close()


# ------------------------------------------------------------------ graphs, streams, waits

def calls_of(kv, seed):
    """Each operator on its own state: (name, run(stream), outputs)."""
    made = []
    c, bt, lens, rng = tl.window_case(kv, [300, 17, 90], 60, 5, seed)
    q, _ = lh.query(rng, 3)
    n = pkv.pkv_decode_window_workspace_bytes(3, bt.shape[1], 60, 5, 2)
    s = dict(c=c, q=q, bt=lh.dev(bt), lens=lh.dev(lens), ws=tl.ws_of(n), out=torch.zeros_like(q), err=tl.flag(), n=n,
             blocks=bt.shape[1])
    made.append(("window", s, lambda s, st: pkv.pkv_decode_window(
        s["c"].pool, s["q"], s["bt"], s["blocks"], s["lens"], 3, lh.SCALE, 60, 5, 2, s["ws"], s["n"], s["out"], s["err"], st),
        lambda s: [s["out"]]))
    c, bt, view, lens, starts, prefix, rng = tl.shared_case(kv, [(20, [5, 33, 2]), (3, [7] * 40)], seed + 1)
    q, _ = lh.query(rng, len(lens))
    n = pkv.pkv_decode_shared_workspace_bytes(len(lens), bt.shape[1], 2, 20, 2, 8)
    s = dict(c=c, q=q, bt=lh.dev(bt), lens=lh.dev(lens), ws=tl.ws_of(n), out=torch.zeros_like(q), err=tl.flag(), n=n,
             blocks=bt.shape[1], B=len(lens), starts=lh.dev(starts), prefix=lh.dev(prefix))
    made.append(("shared", s, lambda s, st: pkv.pkv_decode_shared(
        s["c"].pool, s["q"], s["bt"], s["blocks"], s["lens"], s["B"], s["starts"], s["prefix"], 2, 20, lh.SCALE, 2, 8, s["ws"],
        s["n"], s["out"], s["err"], st), lambda s: [s["out"]]))
    c, bt, lens, rng = tl.whole_case(kv, [300, 17, 90], seed + 2)
    q, _ = lh.query(rng, 3)
    n = pkv.pkv_decode_scored_workspace_bytes(3, bt.shape[1], 4)
    acc = torch.zeros((3, HKV, bt.shape[1] * PS), device="cuda")
    s = dict(c=c, q=q, bt=lh.dev(bt), lens=lh.dev(lens), ws=tl.ws_of(n), out=torch.zeros_like(q), err=tl.flag(), n=n,
             blocks=bt.shape[1], acc=acc, acc_out=torch.zeros_like(acc))
    made.append(("scored", s, lambda s, st: pkv.pkv_decode_scored(
        s["c"].pool, s["q"], s["bt"], s["blocks"], s["lens"], 3, lh.SCALE, s["acc"], s["acc_out"], s["acc"].shape[-1], 4,
        s["ws"], s["n"], s["out"], s["err"], st), lambda s: [s["out"], s["acc_out"]]))
    lens = np.array([300, 17, 90], dtype=np.int32)
    bt, m = lh.shuffled_tables(rng, -(-lens // PS), 19)
    dst, m2 = lh.shuffled_tables(rng, -(-np.minimum(lens, 40) // PS), 3, m)
    c = lh.Cache(kv, m + m2)
    c.host[:] = rng.integers(0, 256, c.host.nbytes, dtype=np.uint8).view(c.host.dtype)
    c.upload()
    acc = lh.dev(tl.acc_of(rng, (3, HKV, 19 * PS), "real"))
    s = dict(c=c, bt=lh.dev(bt), lens=lh.dev(lens), dst=lh.dev(dst), acc=acc, out=torch.zeros((3, HKV, 48), device="cuda"),
             kept=torch.zeros((3, HKV, 40), dtype=torch.int32, device="cuda"), after=torch.zeros(3, dtype=torch.int32, device="cuda"),
             err=tl.flag(), q=acc)
    made.append(("evict", s, lambda s, st: pkv.pkv_evict(
        s["c"].pool, s["bt"], 19, s["lens"], 3, s["dst"], 3, 40, 8, 2, s["acc"], 19 * PS, s["out"], 48, s["kept"], s["after"],
        None, 0, s["err"], st), lambda s: [s["out"], s["kept"], s["after"], s["c"].slab]))
    return made


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("which", range(4))
def test_captured_and_replayed(kv, which):
    name, s, run, outputs = calls_of(kv, 50)[which]
    run(s, None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):                        # launches that follow each other within the graph
            run(s, None)
    for seed in (1, 2):
        gen = torch.Generator("cuda").manual_seed(seed)
        s["q"].copy_(torch.randn(s["q"].shape, generator=gen, device="cuda"))   # the queries, or the weights
        run(s, None)
        torch.cuda.synchronize()
        want = [t.clone() for t in outputs(s)]
        for t in outputs(s):
            if t is not s["c"].slab:
                t.zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outputs(s))), name
    assert pkv.pkv_check_device_error(s["err"]) == (pkv.PKV_OK, 0)


@pytest.mark.parametrize("kv", KV)
def test_two_streams_at_once(kv):
    sides = [calls_of(kv, 60), calls_of(kv, 70)]
    wants = []
    for side in sides:
        for _, s, run, outputs in side:
            run(s, None)
        torch.cuda.synchronize()
        wants.append([[t.clone() for t in outputs(s)] for _, s, _, outputs in side])
    streams = [torch.cuda.Stream() for _ in sides]
    for _ in range(20):
        for side, st in zip(sides, streams):
            for _, s, run, _ in side:
                run(s, st)
    torch.cuda.synchronize()
    for side, want in zip(sides, wants):
        for (name, s, _, outputs), w in zip(side, want):
            assert all(torch.equal(a, b) for a, b in zip(w, outputs(s))), name
            assert pkv.pkv_check_device_error(s["err"]) == (pkv.PKV_OK, 0)


@pytest.mark.parametrize("kv", KV)
def test_waits_that_give_up_are_reported(kv):
    """The testing aid makes waits give up at once: the flag says so, sequences that the waits do not
    concern are computed as usual, and the next call is whole again."""
    lens = [300, 17, 90]
    c, bt, lens, rng = tl.whole_case(kv, lens, 80)
    q, _ = lh.query(rng, 3)
    B, blocks = bt.shape
    acc = torch.zeros((B, HKV, blocks * PS), device="cuda")
    n = max(pkv.pkv_decode_window_workspace_bytes(B, blocks, 100, 3, 2), pkv.pkv_decode_scored_workspace_bytes(B, blocks, 2))
    for call in ("window", "scored"):
        ws = tl.ws_of(n)
        outs = []
        for options in (0, pkv.PKV_STEP_TEST_EXPIRE_WAIT, 0):
            out, err, acc_out = torch.zeros_like(q), tl.flag(), torch.zeros_like(acc)
            if call == "window":
                pkv.pkv_decode_window(c.pool, q, lh.dev(bt), blocks, lh.dev(lens), B, lh.SCALE, 100, 3, 2, ws, n, out, err, None,
                                      options)
            else:
                pkv.pkv_decode_scored(c.pool, q, lh.dev(bt), blocks, lh.dev(lens), B, lh.SCALE, acc, acc_out, blocks * PS, 2,
                                      ws, n, out, err, None, options)
            st, bits = pkv.pkv_check_device_error(err)
            assert bits == (pkv.PKV_DEVERR_TIMEOUT if options else 0)
            outs.append((out, acc_out))
        assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[2]))
        assert all(torch.equal(a[1:], b[1:]) for a, b in zip(outs[0], outs[1]))
    c.close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("groups", [[(40, [5, 33, 2, 9])], [(24, [3] * 70), (30, [4, 6])]])
def test_prefix_waits_that_give_up_end(kv, groups):
    c, bt, view, lens, starts, prefix, rng = tl.shared_case(kv, groups, 90)
    q, _ = lh.query(rng, len(lens))
    want, _ = tl.run_shared(c, bt, lens, starts, prefix, q, 2, 16)
    _, bits = tl.run_shared(c, bt, lens, starts, prefix, q, 2, 16, pkv.PKV_STEP_TEST_EXPIRE_WAIT, ok=False)
    assert bits == pkv.PKV_DEVERR_TIMEOUT
    again, _ = tl.run_shared(c, bt, lens, starts, prefix, q, 2, 16)
    assert torch.equal(want, again)
    c.close()


@pytest.mark.parametrize("kv", KV)
def test_offsets_past_32_bits(kv):
    """Pages whose bytes lie past 4 GiB of the slab."""
    page = pkv.PKV_PAGE_BYTES if kv == "bf16" else pkv.PKV_PAGE_BYTES_FP8
    pages = (5 << 30) // page
    rng = np.random.default_rng(2)
    small = lh.Cache(kv, 24)
    lens = np.array([100, 37], dtype=np.int32)
    local, n = lh.shuffled_tables(rng, -(-lens // PS), 7)
    for b, L in enumerate(lens):
        lh.fill(small, local[b], range(int(L)), rng)
    slab = torch.zeros(pages * page, dtype=torch.uint8, device="cuda")
    base = pages - 24
    slab[base * page:] = torch.from_numpy(small.host.view(np.uint8)).cuda()
    make = pkv.pkv_pool_create if kv == "bf16" else pkv.pkv_pool_create_fp8
    pool = make(slab, slab.numel())
    bt = np.where(local >= 0, local + base, -1).astype(np.int32)
    big = lh.Cache.__new__(lh.Cache)
    big.kv, big.pool, big.slab = kv, pool, slab
    q, qf = lh.query(rng, 2)
    outs = [tl.run_window(big, bt, lens, q, 200, 0, 2), tl.run_scored(big, bt, lens, q, *[torch.zeros((2, HKV, 7 * PS), device="cuda")] * 2, 2)[0],
            tl.run_shared(big, bt, lens, np.array([0, 1, 2], np.int32), np.array([5, 2], np.int32), q, 2, 8)[0]]
    for b, L in enumerate(lens):
        K, V = small.rows(local[b], range(int(L)))
        want, off, _, _ = lh.attend(qf[b], K, V, kv, 2.0 ** -8)
        for o in outs:
            tl.close(o[b], want, off, b)
    dst = np.array([[base + 20, base + 21], [3, 4]], dtype=np.int32)
    acc = tl.acc_of(rng, (2, HKV, 7 * PS), "real")
    _, kept, _, _ = tl.run_evict(big, bt, lens, dst, acc, 32, 4, 1)
    host = torch.cat([slab[3 * page:5 * page], slab[(base + 20) * page:(base + 22) * page]]).cpu().numpy()
    got = lh.Cache(kv, 4)
    got.host[:] = host.view(got.host.dtype)
    for b, table in enumerate(([2, 3], [0, 1])):
        for g in range(HKV):
            K, V = small.rows(local[b], kept[b, g])
            gk, gv = got.rows(table, range(32), got.host)
            assert np.array_equal(gk[g], K[g]) and np.array_equal(gv[g], V[g])
    pkv.pkv_pool_destroy(pool)
