"""Causal attention of chunks against plain attention in 64 bits.  Unused slots of every pool hold NaN,
table entries that no call may read are -1, outputs start as a sentinel; tolerances are those of
``chunk_helpers.attend``."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import chunk_helpers as ch
from tests import long_helpers as lh
from tests import paged_helpers as ph

pytestmark = pytest.mark.gpu

PS, HKV, HQ, D = lh.PS, lh.HKV, lh.HQ, lh.D
KV = ["bf16", "fp8"]


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


SIZES = [
    [(0, 1)], [(0, 2)], [(0, 17)], [(15, 1)], [(16, 1)], [(5, 1), (0, 0), (16, 16), (15, 33)],
    [(100, 64), (300, 1), (127, 1), (128, 1), (126, 3)], [(0, 200)], [(250, 70), (0, 130), (33, 0), (0, 31), (0, 32), (0, 33)],
    [(700, 3)], [(1500, 1), (40, 65)], [(383, 129)], [(0, 1)] * 70, [(900, 40), (0, 0), (0, 0)],
]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_sizes(kv, case):
    b = ch.Batch(kv, SIZES[case], seed=case, pad=case % 3).upload().call()
    assert b.flag() == 0
    b.check().close()


WINDOWS = [
    ([(0, 1)], 1, 0), ([(40, 20)], 1, 0), ([(100, 40), (3, 50)], 16, 5), ([(300, 70)], 17, 16), ([(257, 33), (0, 5)], 50, 33),
    ([(400, 100)], 100, 3), ([(200, 20)], 1000, 8), ([(600, 140), (1000, 1)], 129, 1), ([(90, 64)], 40, 60),
    ([(130, 131)], 2**31 - 1, 2**31 - 1), ([(500, 40)], 100, 2**31 - 1), ([(700, 64)], 333, 0), ([(1000, 3)], 128, 128),
]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("case", range(len(WINDOWS)))
def test_windows(kv, case):
    sizes, window, sinks = WINDOWS[case]
    b = ch.Batch(kv, sizes, window, sinks, seed=50 + case, pad=case % 2).upload().call()
    assert b.flag() == 0
    b.check().close()


@pytest.mark.parametrize("kv", KV)
def test_single_tokens_match_a_decode_step(kv):
    sizes = [(299, 1), (0, 1), (16, 1), (77, 1)]
    b = ch.Batch(kv, sizes, seed=3).upload().call()
    ws = torch.zeros(pkv.pkv_decode_workspace_bytes(4, b.blocks, 4), dtype=torch.uint8, device="cuda")
    ref = torch.empty_like(b.out)
    pkv.pkv_decode_attention(b.cache.pool, b.q, b.dev["bt"], b.blocks, b.dev["lens"], 4, lh.SCALE, 4, ws, ws.numel(), ref)
    assert b.flag() == 0
    b.check()
    b.check(out=ref)
    b.close()


def poison(b, row, tokens, what):
    """Keys and values of some tokens of a row that are not numbers."""
    for t in tokens:
        page, slot = b.bt[row, t // PS], t % PS
        if b.kv == "bf16":
            ph.pool_view(b.cache.host)[page, :, :, slot] = lh.bf16_bits(np.float32(what))
        else:
            for i in range(2):
                for h in range(HKV):
                    b.cache.f8.set_row(page, i, h, slot, np.full(D, 0x7F, np.uint8), np.float32(what))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 3)])
def test_what_is_masked_has_no_effect(kv, what, window, sinks):
    """Tokens that are not finite reach those that attend to them, and no other."""
    sizes = [(200, 90), (0, 150), (150, 2)]
    b = ch.Batch(kv, sizes, window, sinks, seed=8)
    bad = {0: [250, 251, 289], 1: [0, 100], 2: [151]}
    clean = ch.Batch(kv, sizes, window, sinks, seed=8)
    for row, tokens in bad.items():
        poison(b, row, tokens, what)
    b.upload().call()
    clean.upload().call()
    assert b.flag() == clean.flag() == 0
    clean.check()
    got, ref = lh.bf16_values(b.out), lh.bf16_values(clean.out)
    for row, (c, n) in enumerate(sizes):
        for i in range(n):
            t = b.starts[row] + i
            reached = np.isin(bad[row], ch.seen(c + i, window, sinks)).any()
            if reached:
                assert not np.isfinite(got[t]).any(), (row, i)
            else:
                assert np.array_equal(got[t], ref[t]), (row, i)
    b.close()
    clean.close()


@pytest.mark.parametrize("window", [0, 40])
def test_values_that_are_not_finite_stay_in_their_dimension(window):
    """(BF16 pages: a row of codes has one scale.)"""
    sizes = [(100, 60)]
    b, clean = (ch.Batch("bf16", sizes, window, 0, seed=9) for _ in range(2))
    P = ph.pool_view(b.cache.host)
    for t, d in ((130, 5), (150, 63)):
        P[b.bt[0, t // PS], 1, 3, t % PS, d] = lh.bf16_bits([np.inf])[0]
    b.upload().call()
    clean.upload().call()
    got, ref = lh.bf16_values(b.out), lh.bf16_values(clean.out)
    for i in range(60):
        hit = [d for t, d in ((130, 5), (150, 63)) if t in ch.seen(100 + i, window, 0)]
        want = ref[i].copy()
        keep = np.ones((HQ, D), bool)
        keep[12:16, hit] = False
        assert np.array_equal(got[i][keep], want[keep]) and not np.isfinite(got[i][~keep]).any()
    b.close()
    clean.close()


@pytest.mark.parametrize("kv", KV)
def test_scores_far_apart(kv):
    """Rows whose largest score comes late, by far more than the exponent's range."""
    b = ch.Batch(kv, [(300, 40), (0, 100)], seed=10)
    # keys that grow along the sequence, and queries along one of them
    for row, (c, n) in enumerate(b.sizes):
        for t in b.tokens[row]:
            k, v = b.rng.standard_normal((2, HKV, D))
            b.cache.put(b.bt[row, t // PS], t % PS, k * (0.01 + t / 4.0), v)
    b.upload().call()
    assert b.flag() == 0
    b.check().close()


@pytest.mark.parametrize("kv", KV)
def test_equal_scores_and_large_values(kv):
    b = ch.Batch(kv, [(70, 40)], seed=11)
    for t in b.tokens[0]:
        v = b.rng.standard_normal((HKV, D)) * (2.0 ** 40 if t % 7 == 0 else 1.0)
        b.cache.put(b.bt[0, t // PS], t % PS, np.ones((HKV, D)), v)
    b.upload().call()
    assert b.flag() == 0
    b.check().close()


@pytest.mark.parametrize("kv", KV)
def test_device_checks(kv):
    sizes = [(40, 5), (100, 30), (10, 3), (0, 40), (60, 2), (20, 4)]
    b = ch.Batch(kv, sizes, seed=12, blocks=9, spare=1)
    b.lens[2] = 2                              # shorter than its new tokens
    b.lens[4] = 9 * PS + 1                     # longer than the table
    b.bt[3, 1] = 10 ** 6                       # a page outside the pool
    b.upload().call()
    assert b.flag() == pkv.PKV_DEVERR_LENGTH | pkv.PKV_DEVERR_PAGE_RANGE
    b.check(rows=[0, 1, 5])
    got = b.out.float().cpu().numpy()
    for row in (2, 4):
        assert not got[b.starts[row]:b.starts[row + 1]].any()
    assert not got[b.starts[3] + 16:b.starts[4]].any()      # (those that attend to the bad page)
    b.close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("starts", [[0, 5, 3, 20], [0, -4, 6, 20], [0, 5, 9, 21], [3, 5, 9, 20]])
def test_bad_starts_are_reported(kv, starts):
    b = ch.Batch(kv, [(30, 5), (30, 4), (30, 11)], seed=13)
    b.starts = np.array(starts, np.int32)
    b.upload().call()
    assert b.flag() == pkv.PKV_DEVERR_LENGTH
    b.close()


@pytest.mark.parametrize("kv", KV)
def test_same_bits_again_and_on_another_stream(kv):
    sizes = [(2000, 1), (500, 130), (0, 64), (3, 7), (900, 0), (1200, 33)]
    b = ch.Batch(kv, sizes, seed=14, pad=9).upload().call()
    assert b.flag() == 0
    first = b.out.clone()
    side = torch.cuda.Stream()
    for stream in (None, side):
        b.out.fill_(ch.SENTINEL)
        torch.cuda.synchronize()
        b.call(stream)
        assert b.flag() == 0 and torch.equal(b.out, first)
    b.check().close()


@pytest.mark.parametrize("kv", KV)
def test_captured_and_replayed_with_other_sizes(kv):
    """One graph, replayed with other lengths and counts in its arrays."""
    a = ch.Batch(kv, [(100, 40), (0, 70), (300, 1)], seed=15, blocks=64, spare=100).upload().call()
    assert a.flag() == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call()
    a.out.fill_(ch.SENTINEL)
    g.replay()
    assert a.flag() == 0
    a.check()
    other = ch.Batch(kv, [(17, 1), (600, 100), (0, 9)], seed=16, blocks=64, pad=1)
    assert other.T == a.T and other.cache.pages <= a.cache.pages
    other.upload()
    a.cache.slab[:other.cache.slab.numel()].copy_(other.cache.slab)
    for x in ("bt", "lens", "starts"):
        a.dev[x].copy_(other.dev[x])
    a.q.copy_(other.q)
    a.out.fill_(ch.SENTINEL)
    g.replay()
    assert a.flag() == 0
    other.check(out=a.out)
    a.close()
    other.close()


def exact_rows(slab, kv, pages, L):
    """K, V [8][L][64] in FP64 on the GPU of a sequence with the given pages."""
    if kv == "bf16":
        x = slab.view(torch.bfloat16).view(-1, 2, HKV, PS, D)[pages].double()
        return (x[:, i].transpose(0, 1).reshape(HKV, -1, D)[:, :L] for i in (0, 1))
    import oracle

    unit = oracle.FP8_PAGE_BYTES // HKV
    u = slab.view(-1, HKV, unit)[pages]
    sc = u[..., 2 * PS * D:].contiguous().view(torch.float32).view(-1, HKV, 2, PS).double()
    k = u[..., :PS * D].contiguous().view(torch.float8_e4m3fn).double().view(-1, HKV, PS, D) * sc[:, :, 0, :, None]
    s, d = np.arange(PS)[:, None], np.arange(D)[None, :]
    off = (s // 2) * 2 * D + ((d // 8) ^ ((2 * (s // 2)) % 8)) * 16 + (d % 8) * 2 + s % 2
    v = u[..., PS * D + torch.from_numpy(off.reshape(-1)).cuda()].contiguous().view(torch.float8_e4m3fn).double()
    v = v.view(-1, HKV, PS, D) * sc[:, :, 1, :, None]
    return (x.transpose(0, 1).reshape(HKV, -1, D)[:, :L] for x in (k, v))


BIG = [
    ([(3000, 500), (4000, 1), (0, 900), (100, 257), (5000, 2)] + [(2500, 1)] * 20, 0, 0),
    ([(0, 2048)] * 3, 0, 0), ([(20000, 64)], 0, 0), ([(20000, 1)], 0, 0), ([(9000, 700), (4000, 33)], 1000, 5),
    ([(i * 7 % 900, i % 5) for i in range(300)], 0, 0), ([(33000, 300)], 0, 0),
    ([(i * 31 % 3000, 1 + i % 3) for i in range(190)], 200, 17),
    ([(i * 13 % 700, i % 3) for i in range(4096)], 0, 0), ([(i * 13 % 90, 1) for i in range(4096)], 30, 2),
]


def check_on_gpu(kv, sizes, window, sinks, case):
    """Long and many sequences: every output row against attention in 64 bits on the GPU.  The bound is
    ``chunk_helpers.attend``'s with the weights' part summed in closed form: off = 2 * 2^-8 * sum p |v| for the
    rounded weights and their sum, 2^-8 |out| for the output, 2^-12 sum p |v| for the scores (|s| < 2^7, off by
    at most 2^-18 of the products' absolute sum, itself below 2^6 here, as is checked)."""
    rng = np.random.default_rng(case)
    lens = np.array([c + n for c, n in sizes])
    need = -(-lens // PS)
    pages = int(need.sum())
    gen = torch.Generator("cuda").manual_seed(case)
    x = torch.randn((pages, 2, HKV, PS, D), generator=gen, device="cuda").to(torch.bfloat16)
    if kv == "bf16":
        slab = x.view(torch.uint8).view(-1)
        pool = pkv.pkv_pool_create(slab, slab.numel())
    else:
        slab = torch.zeros(pages * pkv.PKV_PAGE_BYTES_FP8, dtype=torch.uint8, device="cuda")
        pool = pkv.pkv_pool_create_fp8(slab, slab.numel())
        slots = torch.arange(pages * PS, device="cuda")
        rows = x.permute(1, 0, 3, 2, 4).reshape(2, -1, HKV, D).contiguous()
        pkv.pkv_chunk_append(pool, rows[0], 512, rows[1], 512, None, 0, None, None, None, 0.0, slots,
                             torch.zeros(pages * PS, dtype=torch.int32, device="cuda"), 0, None, pages * PS,
                             pkv.rope_table(16, "cuda"), 16)
    bt, _ = lh.shuffled_tables(rng, need, int(need.max()))
    starts = np.concatenate([[0], np.cumsum([n for _, n in sizes])]).astype(np.int32)
    T, B = int(starts[-1]), len(sizes)
    q = torch.randn((T, HQ, D), generator=gen, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, ch.SENTINEL)
    nbytes = pkv.pkv_chunk_attention_workspace_bytes(B, T)
    ws, err = torch.zeros(nbytes, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    btd = lh.dev(bt)
    pkv.pkv_chunk_attention(pool, q, btd, bt.shape[1], lh.dev(lens.astype(np.int32)), lh.dev(starts), B, T, lh.SCALE, window,
                            sinks, ws, nbytes, out, err)
    assert int(err) == 0
    for b, (c, n) in enumerate(sizes):
        if not n or (B > 1000 and b % 61 and b < B - 2):
            continue
        L = c + n
        K, V = exact_rows(slab, kv, btd[b, :int(need[b])].long(), L)
        p = torch.arange(c, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None, :]
        hidden = j > p
        if window:
            hidden |= (j <= p - window) & (j >= sinks)
        for h in range(HQ):
            qh = q[starts[b]:starts[b + 1], h].double()
            s = qh @ K[h // 4].T * lh.SCALE
            assert float(s.abs().max()) < 64 and float((qh.abs() @ K[h // 4].abs().T).max()) * lh.SCALE < 64
            w = torch.softmax(s.masked_fill(hidden, -torch.inf), -1)
            want, mass = w @ V[h // 4], w @ V[h // 4].abs()
            off = (2.0 ** -7 + 2.0 ** -11) * mass + 2.0 ** -8 * want.abs() + 2.0 ** -20
            bad = ~((out[starts[b]:starts[b + 1], h].double() - want).abs() <= off)
            assert not bad.any(), (b, h, bad.nonzero()[:4].tolist())
    pkv.pkv_pool_destroy(pool)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("case", range(len(BIG)))
def test_large_batches(kv, case):
    check_on_gpu(kv, *BIG[case], case)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("seed", range(16))
def test_random_batches(kv, seed):
    """Batches of 1 to 60 sequences: chunks, single tokens and nothing, fresh and continued, with and without windows."""
    r = np.random.default_rng(1000 + seed)
    B = int(np.exp(r.uniform(0, np.log(60))))
    cached = np.exp(r.uniform(0, np.log(4000), B)).astype(int) * (r.random(B) < 0.8)
    new = np.where(r.random(B) < r.random(), 1, np.exp(r.uniform(0, np.log(600), B)).astype(int)) * (r.random(B) < 0.9)
    new[int(r.integers(0, B))] += 1
    window = int(np.exp(r.uniform(0, np.log(1500)))) if r.random() < 0.5 else 0
    check_on_gpu(kv, list(zip(cached.tolist(), new.tolist())), window, int(r.integers(0, 200)) if window else 0, seed)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("B,T", [(1, 2), (2, 3), (2, 4), (7, 13), (7, 14), (8, 15), (8, 16), (31, 61), (31, 62), (32, 64)])
def test_either_way_of_sharing_out_single_tokens(kv, B, T):
    """Tokens a sequence next to where single tokens get a kernel of their own, in arrays of T with and without padding."""
    rng = np.random.default_rng(B * 100 + T)
    for full in (True, False):
        new = np.ones(B, int)
        new[rng.integers(0, B)] += (T - B if full else (T - B) // 2)
        b = ch.Batch(kv, [(int(rng.integers(0, 150)), int(n)) for n in new], seed=T, pad=T - int(new.sum())).upload().call()
        assert b.flag() == 0
        b.check().close()


@pytest.mark.parametrize("kv", KV)
def test_same_bits_without_programmatic_launches(kv):
    sizes = [(600, 40)] + [(i * 17 % 300, 1 + i % 2) for i in range(40)]
    b = ch.Batch(kv, sizes, seed=41).upload().call()
    assert b.flag() == 0
    first = b.out.clone()
    b.out.fill_(ch.SENTINEL)
    torch.cuda.synchronize()
    for _ in range(3):
        b.call(options=pkv.PKV_STEP_NO_PDL)
    assert b.flag() == 0 and torch.equal(b.out, first)
    b.check(rows=range(0, 41, 7)).close()


@pytest.mark.parametrize("kv", KV)
def test_pages_that_sequences_share(kv):
    """Two sequences behind the same first pages, one of which is also named twice by one table."""
    b = ch.Batch(kv, [(100, 40), (100, 1), (90, 17)], seed=51)
    b.bt[1, :6] = b.bt[0, :6]
    b.bt[2, 1] = b.bt[2, 0]
    b.upload().call()
    assert b.flag() == 0
    b.check().close()
