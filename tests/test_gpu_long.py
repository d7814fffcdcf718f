"""GPU parity of the long-context operators against plain implementations in 64 bits.

Unused slots of every pool hold NaN, table entries that no call may read are -1 or name pages of
NaN, and outputs start as a sentinel.  Tolerances are those of ``long_helpers.attend``."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
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


def flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def ws_of(nbytes):
    return torch.zeros(max(nbytes, 16), dtype=torch.uint8, device="cuda")


def close(got, want, off, what=""):
    got = lh.bf16_values(got)
    bad = ~(np.abs(got - want) <= off)
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], off[bad][:4])


# ------------------------------------------------------------------ window

def visible(L, window, sinks):
    return [t for t in range(L) if t < sinks or t >= L - window]


def window_case(kv, lens, window, sinks, seed, blocks=None):
    """Only visible tokens have rows; pages without one are -1 in the table."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int32)
    need = -(-lens // PS)
    blocks = blocks or int(need.max())
    live = [sorted({t // PS for t in visible(int(L), window, sinks)}) for L in lens]
    n = sum(map(len, live))
    ids = rng.permutation(n)
    bt = np.full((lens.size, blocks), -1, dtype=np.int32)
    at = 0
    for b, pages in enumerate(live):
        bt[b, pages] = ids[at:at + len(pages)]
        at += len(pages)
    c = lh.Cache(kv, n)
    for b, L in enumerate(lens):
        lh.fill(c, bt[b], visible(int(L), window, sinks), rng)
    return c.upload(), bt, lens, rng


def run_window(c, bt, lens, q, window, sinks, ppc=0, options=0, out=None, stream=None):
    B, blocks = bt.shape
    nbytes = pkv.pkv_decode_window_workspace_bytes(B, blocks, window, sinks, ppc)
    ws, err = ws_of(nbytes), flag()
    out = torch.full((B, HQ, D), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    pkv.pkv_decode_window(c.pool, q, lh.dev(bt), blocks, lh.dev(lens), B, lh.SCALE, window, sinks, ppc, ws, nbytes, out,
                          err, stream, options)
    assert pkv.pkv_check_device_error(err, stream) == (pkv.PKV_OK, 0)
    assert not ws[:B * HKV * 4].any() or blocks <= max(ppc, 1)   # the merge counters are zero again
    return out


WINDOWS = [
    ([1], 1, 0), ([1, 2, 15, 16, 17, 31, 33], 1, 0), ([1, 5, 16, 40, 100], 7, 3), ([300, 17, 64, 1], 16, 16),
    ([300, 301, 315, 320, 321], 17, 5), ([257, 90, 33], 50, 33), ([200, 20, 35], 1000, 8), ([130, 131], 129, 1),
    ([90, 91, 92, 93], 40, 60), ([700, 650, 3], 333, 0), ([2048, 48], 2**31 - 1, 2**31 - 1), ([500, 40], 100, 2**31 - 1),
]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("case", range(len(WINDOWS)))
def test_window(kv, case):
    lens, window, sinks = WINDOWS[case]
    c, bt, lens, rng = window_case(kv, lens, window, sinks, 100 + case)
    q, qf = lh.query(rng, len(lens))
    outs = [run_window(c, bt, lens, q, window, sinks, ppc) for ppc in (0, 1, 3, 16, 128)]
    for b, L in enumerate(lens):
        K, V = c.rows(bt[b], visible(int(L), window, sinks))
        want, off, _, _ = lh.attend(qf[b], K, V, kv)
        for o in outs:
            close(o[b], want, off, (b, L))
    c.close()


@pytest.mark.parametrize("kv", KV)
def test_window_options_and_batches_keep_every_bit(kv):
    lens = [900, 1, 40, 333, 16, 600]
    c, bt, lens, rng = window_case(kv, lens, 250, 20, 7, blocks=80)
    q, _ = lh.query(rng, len(lens))
    ref = run_window(c, bt, lens, q, 250, 20, 4)
    for options in (pkv.PKV_STEP_SORTED, pkv.PKV_STEP_NO_PDL, pkv.PKV_STEP_RING(3), pkv.PKV_STEP_RING(4),
                    pkv.PKV_DECODE_MMA | pkv.PKV_STEP_RING(2) | pkv.PKV_STEP_SORTED):
        assert torch.equal(run_window(c, bt, lens, q, 250, 20, 4, options), ref), hex(options)
    for b in range(len(lens)):
        one = run_window(c, bt[b:b + 1], lens[b:b + 1], q[b:b + 1], 250, 20, 4)
        assert torch.equal(one[0], ref[b])
    # a window over everything is the attention over everything
    c.close()


@pytest.mark.parametrize("kv", KV)
def test_window_over_everything_is_decode_attention(kv):
    c, bt, lens, rng = window_case(kv, [300, 77, 16, 1], 300, 0, 9)
    q, _ = lh.query(rng, 4)
    out = run_window(c, bt, lens, q, 300, 0, 4)
    ws = ws_of(pkv.pkv_decode_workspace_bytes(4, bt.shape[1], 4))
    ref = torch.empty_like(out)
    pkv.pkv_decode_attention(c.pool, q, lh.dev(bt), bt.shape[1], lh.dev(lens), 4, lh.SCALE, 4, ws, ws.numel(), ref)
    assert torch.equal(out, ref)
    c.close()


@pytest.mark.parametrize("kv", KV)
def test_window_device_checks(kv):
    c, bt, lens, rng = window_case(kv, [100, 50, 40], 20, 2, 11, blocks=7)
    q, qf = lh.query(rng, 3)
    lens2, bt2 = lens.copy(), bt.copy()
    lens2[1] = 7 * PS + 1                        # beyond the table
    bt2[0, 3] = -7                               # never looked up: no token of page 3 is visible
    bt2[2, 2] = 10 ** 6                          # the newest page
    B, blocks = bt.shape
    nbytes = pkv.pkv_decode_window_workspace_bytes(B, blocks, 20, 2, 128)
    ws, err, out = ws_of(nbytes), flag(), torch.full((B, HQ, D), 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.pkv_decode_window(c.pool, q, lh.dev(bt2), blocks, lh.dev(lens2), B, lh.SCALE, 20, 2, 128, ws, nbytes, out, err)
    st, bits = pkv.pkv_check_device_error(err)
    assert st == pkv.PKV_ERR_DEVICE_BOUNDS and bits == pkv.PKV_DEVERR_LENGTH | pkv.PKV_DEVERR_PAGE_RANGE
    assert not out[1].any() and not out[2].any()
    K, V = c.rows(bt[0], visible(100, 20, 2))
    close(out[0], *lh.attend(qf[0], K, V, kv)[:2])
    # no error flag, and lengths that are not one
    lens2[:] = [0, -5, -2**31]
    out.fill_(7.0)
    pkv.pkv_decode_window(c.pool, q, lh.dev(bt), blocks, lh.dev(lens2), B, lh.SCALE, 20, 2, 128, ws, nbytes, out, None)
    torch.cuda.synchronize()
    assert not out.any()
    c.close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 4), (60, 16), (500, 0)])
def test_step_window_is_append_then_window(kv, window, sinks):
    lens = [100, 33, 1, 16, 17, 64]
    c, bt, lens, rng = window_case(kv, lens, window, sinks, 21)
    B, blocks = bt.shape
    q, _ = lh.query(rng, B)
    kn, vn = (torch.from_numpy(lh.bf16_bits(rng.standard_normal((B, HKV, D))).view(np.int16).copy())
              .view(torch.bfloat16).cuda() for _ in range(2))
    rope = pkv.rope_table(128, "cuda")
    start = c.slab.clone()
    nbytes = pkv.pkv_decode_window_workspace_bytes(B, blocks, window, sinks, 2)
    ws, err = ws_of(nbytes), flag()
    btd, ld = lh.dev(bt), lh.dev(lens)
    q1, out1 = q.clone(), torch.empty_like(q)
    pkv.pkv_append_rope(c.pool, kn, vn, q1, btd, blocks, ld - 1, B, rope, 128, err)
    pkv.pkv_decode_window(c.pool, q1, btd, blocks, ld, B, lh.SCALE, window, sinks, 2, ws, nbytes, out1, err)
    slab1 = c.slab.clone()
    c.slab.copy_(start)
    q2, out2 = q.clone(), torch.empty_like(q)
    pkv.pkv_decode_step_window(c.pool, kn, vn, q2, btd, blocks, ld, B, rope, 128, lh.SCALE, window, sinks, 2, ws, nbytes,
                               out2, err)
    assert pkv.pkv_check_device_error(err) == (pkv.PKV_OK, 0)
    assert torch.equal(out1, out2) and torch.equal(q1, q2) and torch.equal(slab1, c.slab)
    assert not torch.equal(start, slab1)
    c.close()


# ------------------------------------------------------------------ shared prefix

def shared_case(kv, groups, seed, extra_blocks=0):
    """groups: [(prefix pages, [own tokens of each sequence])].  The first entries of the rows of
    all but a group's first sequence are -1: they are not read."""
    rng = np.random.default_rng(seed)
    own = [n for _, ns in groups for n in ns]
    of = [i for i, (_, ns) in enumerate(groups) for _ in ns]
    prefix = np.array([p for p, _ in groups], dtype=np.int32)
    starts = np.concatenate([[0], np.cumsum([len(ns) for _, ns in groups])]).astype(np.int32)
    blocks = max(max(prefix[g] + -(-n // PS) for g, n in zip(of, own)), 1) + extra_blocks
    pages = int(prefix.sum()) + sum(-(-n // PS) for n in own)
    ids = iter(rng.permutation(max(pages, 1)).tolist())
    c = lh.Cache(kv, max(pages, 1))
    bt = np.full((len(own), blocks), -1, dtype=np.int32)
    view = bt.copy()                              # what the sequences see
    for g, (p, ns) in enumerate(groups):
        row = [next(ids) for _ in range(p)]
        bt[starts[g], :p] = row
        lh.fill(c, np.array(row + [0]), range(p * PS), rng)
        for b in range(starts[g], starts[g + 1]):
            view[b, :p] = row
            n = -(-own[b] // PS)
            bt[b, p:p + n] = view[b, p:p + n] = [next(ids) for _ in range(n)]
            lh.fill(c, view[b], range(p * PS, p * PS + own[b]), rng)
    lens = np.array([prefix[g] * PS + n for g, n in zip(of, own)], dtype=np.int32)
    return c.upload(), bt, view, lens, starts, prefix, rng


def run_shared(c, bt, lens, starts, prefix, q, ppc=0, pppc=0, options=0, max_prefix=None, ok=True, stream=None):
    B, blocks = bt.shape
    G = len(prefix)
    mp = int(prefix.max()) if max_prefix is None else max_prefix
    nbytes = pkv.pkv_decode_shared_workspace_bytes(B, blocks, G, mp, ppc, pppc)
    ws, err = ws_of(nbytes), flag()
    out = torch.full((B, HQ, D), 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.pkv_decode_shared(c.pool, q, lh.dev(bt), blocks, lh.dev(lens), B, lh.dev(starts), lh.dev(prefix), G, mp,
                          lh.SCALE, ppc, pppc, ws, nbytes, out, err, stream, options)
    st, bits = pkv.pkv_check_device_error(err, stream)
    if ok:
        assert (st, bits) == (pkv.PKV_OK, 0)
        assert not ws[:B * HKV * 4].any()
    return out, bits


SHARED = [
    [(0, [1])], [(1, [1])], [(2, [5, 40])], [(9, [1, 16, 17, 33, 2])], [(3, [20]), (0, [7, 50]), (17, [1, 1, 30])],
    [(8, [10] * 33)], [(16, [3] * 64), (1, [4] * 2)], [(5, [2] * 70)], [(40, [100, 1]), (25, [300])],
    [(7, [0, 16, 0])], [(1, [0])], [(130, [5, 9, 1])],
]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_shared(kv, case):
    c, bt, view, lens, starts, prefix, rng = shared_case(kv, SHARED[case], 200 + case)
    q, qf = lh.query(rng, len(lens))
    outs = [run_shared(c, bt, lens, starts, prefix, q, *a)[0] for a in ((0, 0), (2, 8), (128, 16), (1, 10000))]
    for b, L in enumerate(lens):
        K, V = c.rows(view[b], range(int(L)))
        want, off, _, _ = lh.attend(qf[b], K, V, kv, 2.0 ** -8)
        for o in outs:
            close(o[b], want, off, (b, L))
    c.close()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("scale", [64, 256, 1024])
@pytest.mark.parametrize("groups", [[(130, [5, 9, 1])], [(40, [3] * 40), (25, [30]), (8, [1, 1])]])
def test_shared_scores_far_apart(kv, scale, groups):
    """Long queries: later scores lie hundreds of powers of two above the first ones (at scale 64 some
    rows' do, at 1024 nearly every row's, several times), so the references of rows move, in some rows
    of a tile and not in others."""
    c, bt, view, lens, starts, prefix, rng = shared_case(kv, groups, 220 + scale)
    q, qf = lh.query(rng, len(lens))
    q, qf = q * scale, qf * scale                 # a power of two: exact
    outs = [run_shared(c, bt, lens, starts, prefix, q, *a)[0] for a in ((0, 0), (2, 8), (1, 10000))]
    moved = 0
    for b, L in enumerate(lens):
        K, V = c.rows(view[b], range(int(L)))
        want, off, _, _ = lh.attend(qf[b], K, V, kv, 2.0 ** -8)
        for o in outs:
            close(o[b], want, off, (b, L))
        n = int(prefix[np.searchsorted(starts, b, side="right") - 1]) * PS
        s = np.einsum("hd,hnd->hn", qf[b], np.repeat(K, 4, 0))[:, :n] * (lh.SCALE * np.log2(np.e))
        first = s[:, [t for t in range(min(n, 128)) if t % PS < 8]].max(1)
        moved += int((s.max(1) > first + 70).sum())
    assert moved or scale == 64
    c.close()


@pytest.mark.parametrize("scale", [0.0, 1e-38, 2.0 ** -90])
def test_shared_fp8_values_of_nothing(scale):
    """Prefix tokens whose V row scale is zero or nearly so: they weigh, and add nothing."""
    c, bt, view, lens, starts, prefix, rng = shared_case("fp8", [(17, [5, 33, 1])], 231)
    for t in rng.choice(17 * PS, 120, replace=False):
        c.f8.scales[bt[0, t // PS], 1, :, t % PS] = scale
    c.slab.copy_(torch.from_numpy(c.host).cuda())
    q, qf = lh.query(rng, len(lens))
    out, _ = run_shared(c, bt, lens, starts, prefix, q, 0, 0)
    for b, L in enumerate(lens):
        K, V = c.rows(view[b], range(int(L)))
        want, off, _, _ = lh.attend(qf[b], K, V, "fp8", 2.0 ** -8)
        close(out[b], want, off, (b, L))
    c.close()


@pytest.mark.parametrize("kv", KV)
def test_shared_rows_do_not_depend_on_their_group(kv):
    groups = [(20, [5, 33, 2, 90]), (3, [7]), (0, [40, 1])]
    c, bt, view, lens, starts, prefix, rng = shared_case(kv, groups, 5, extra_blocks=3)
    q, _ = lh.query(rng, len(lens))
    ref, _ = run_shared(c, bt, lens, starts, prefix, q, 2, 8)
    again, _ = run_shared(c, bt, lens, starts, prefix, q, 2, 8, pkv.PKV_STEP_NO_PDL | pkv.PKV_STEP_RING(4))
    assert torch.equal(ref, again)
    looser, _ = run_shared(c, bt, lens, starts, prefix, q, 2, 8, max_prefix=bt.shape[1])
    assert torch.equal(ref, looser)
    for b in range(len(lens)):
        g = int(np.searchsorted(starts, b, side="right")) - 1
        one, _ = run_shared(c, view[b:b + 1], lens[b:b + 1], np.array([0, 1], np.int32), prefix[g:g + 1], q[b:b + 1], 2, 8)
        assert torch.equal(one[0], ref[b]), b
    c.close()


@pytest.mark.parametrize("kv", KV)
def test_shared_device_checks(kv):
    groups = [(2, [5, 6]), (3, [7, 9]), (1, [4]), (2, [8])]
    c, bt, view, lens, starts, prefix, rng = shared_case(kv, groups, 6)
    q, qf = lh.query(rng, len(lens))
    lens2, prefix2, bt2 = lens.copy(), prefix.copy(), bt.copy()
    lens2[1] = 2 * PS - 1                         # shorter than its prefix
    prefix2[1] = 4                                # above the bound of 3
    prefix2[2] = -1
    out, bits = run_shared(c, bt2, lens2, starts, prefix2, q, 128, 8, max_prefix=3, ok=False)
    assert bits == pkv.PKV_DEVERR_LENGTH
    for b in (1, 2, 3, 4):
        assert not out[b].any(), b
    for b in (0, 5):
        K, V = c.rows(view[b], range(int(lens[b])))
        close(out[b], *lh.attend(qf[b], K, V, kv, 2.0 ** -8)[:2])
    # sequences that are in no group; starts that run outside the batch
    for bad in ([0, 2, 4, 5, 5], [1, 2, 4, 5, 6], [-3, 2, 4, 5, 6]):
        out, bits = run_shared(c, bt, lens, np.array(bad, np.int32), prefix, q, 128, 8, ok=False)
        # ([1, ...]: the prefix is looked up in the row of sequence 1, whose first entries are -1)
        assert bits == pkv.PKV_DEVERR_LENGTH | (pkv.PKV_DEVERR_PAGE_RANGE if bad[0] == 1 else 0)
    # a page outside the pool in a prefix and in a sequence's own part
    bt2[0, 1], bt2[5, 2] = 1 << 30, -1
    out, bits = run_shared(c, bt2, lens, starts, prefix, q, 128, 8, ok=False)
    assert bits == pkv.PKV_DEVERR_PAGE_RANGE
    for b in (2, 3, 4):
        K, V = c.rows(view[b], range(int(lens[b])))
        close(out[b], *lh.attend(qf[b], K, V, kv, 2.0 ** -8)[:2])
    c.close()


# ------------------------------------------------------------------ scored

def whole_case(kv, lens, seed, blocks=None):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int32)
    need = -(-lens // PS)
    bt, n = lh.shuffled_tables(rng, need, blocks or max(int(need.max()), 1))
    c = lh.Cache(kv, max(n, 1))
    for b, L in enumerate(lens):
        lh.fill(c, bt[b], range(int(L)), rng)
    return c.upload(), bt, lens, rng


def run_scored(c, bt, lens, q, acc, acc_out, ppc=0, options=0, ok=True):
    B, blocks = bt.shape
    nbytes = pkv.pkv_decode_scored_workspace_bytes(B, blocks, ppc)
    ws, err = ws_of(nbytes), flag()
    ws[B * HKV * 4 + 256:] = 0xFF                 # stale scores are NaN
    out = torch.full((B, HQ, D), 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.pkv_decode_scored(c.pool, q, lh.dev(bt), blocks, lh.dev(lens), B, lh.SCALE, acc, acc_out, acc.shape[-1], ppc, ws,
                          nbytes, out, err, None, options)
    st, bits = pkv.pkv_check_device_error(err)
    if ok:
        assert (st, bits) == (pkv.PKV_OK, 0)
    return out, bits


SCORED = [[1], [16, 1, 17, 15], [300, 5, 64], [1100, 33], [2048, 700, 3, 256]]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("case", range(len(SCORED)))
def test_scored(kv, case):
    c, bt, lens, rng = whole_case(kv, SCORED[case], 300 + case)
    B, n = len(lens), bt.shape[1] * PS
    q, qf = lh.query(rng, B)
    a0 = rng.random((B, HKV, n + 3)).astype(np.float32)
    for ppc in (0, 1, 128):
        acc, acc_out = lh.dev(a0), torch.full((B, HKV, n + 3), -9.0, device="cuda")
        out, _ = run_scored(c, bt, lens, q, acc, acc_out, ppc)
        same = acc.clone()
        out2, _ = run_scored(c, bt, lens, q, same, same, ppc, pkv.PKV_STEP_SORTED)
        assert torch.equal(out, out2) and np.array_equal(acc.cpu().numpy(), a0)
        got, got2 = acc_out.cpu().numpy().astype(np.float64), same.cpu().numpy()
        for b, L in enumerate(lens):
            K, V = c.rows(bt[b], range(int(L)))
            want, off, p, dp = lh.attend(qf[b], K, V, kv)
            close(out[b], want, off, (b, L))
            w = a0[b, :, :L] + p.reshape(HKV, 4, L).sum(1)
            # the weights' own error, the exponential's and four FP32 additions
            tol = dp.reshape(HKV, 4, L).sum(1) + 2.0 ** -20 * p.reshape(HKV, 4, L).sum(1) + 2.0 ** -24 * 4 * w
            assert (np.abs(got[b, :, :L] - w) <= tol).all()
            assert (got[b, :, L:] == -9.0).all()
            assert np.array_equal(got2[b, :, :L], got[b, :, :L].astype(np.float32))
            assert np.array_equal(got2[b, :, L:], a0[b, :, L:])
    c.close()


@pytest.mark.parametrize("kv", KV)
def test_scored_over_a_wide_table_is_the_same(kv):
    """Wide tables (here over 4096 tokens) add the weights in a launch of their own."""
    c, bt, lens, rng = whole_case(kv, [300, 77, 1500, 1], 18)
    q, _ = lh.query(rng, 4)
    wide = np.full((4, 1025), -1, dtype=np.int32)
    wide[:, :bt.shape[1]] = bt
    got = []
    for table in (bt, wide):
        acc = torch.from_numpy(np.random.default_rng(1).random((4, HKV, 1025 * PS), dtype=np.float32)).cuda()
        acc_out = torch.full_like(acc, -9.0)
        out, _ = run_scored(c, table, lens, q, acc, acc_out, 8)
        got.append((out, acc_out))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    c.close()


@pytest.mark.parametrize("offset", [16, 48, 64, 112])
@pytest.mark.parametrize("blocks", [32, 300])      # the weights added in the same launch, in a second one
def test_scored_with_a_workspace_off_the_line(blocks, offset):
    """Scores that do not begin on a cache line: the same results, and nothing around the workspace
    changes, call after call."""
    c, bt, lens, rng = whole_case("bf16", [490, 33, 7], 52)
    B = len(lens)
    q, _ = lh.query(rng, B)
    table = np.full((B, blocks), -1, dtype=np.int32)
    table[:, :min(blocks, bt.shape[1])] = bt[:, :blocks]
    acc = lh.dev(rng.random((B, HKV, blocks * PS)).astype(np.float32))
    want_acc = acc.clone()
    want, _ = run_scored(c, table, lens, q, want_acc, want_acc)
    nbytes = pkv.pkv_decode_scored_workspace_bytes(B, blocks, 0)
    room = torch.full((nbytes + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    start = offset + (-room.data_ptr()) % 128
    ws, err = room[start:start + nbytes], flag()
    ws[:B * HKV * 4] = 0
    for _ in range(3):
        got, out = torch.empty_like(acc), torch.empty_like(want)
        got.copy_(acc)
        pkv.pkv_decode_scored(c.pool, q, lh.dev(table), blocks, lh.dev(lens), B, lh.SCALE, acc, got, acc.shape[-1], 0, ws,
                              nbytes, out, err)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(got, want_acc)
    assert pkv.pkv_check_device_error(err) == (pkv.PKV_OK, 0)
    assert bool((room[:start] == 0x5A).all()) and bool((room[start + nbytes:] == 0x5A).all())


@pytest.mark.parametrize("kv", KV)
def test_scored_output_is_decode_attention(kv):
    """Bit for bit on BF16 pages; on FP8 pages the scores are held more exactly, and both are within
    their distance of the same values."""
    c, bt, lens, rng = whole_case(kv, [300, 77, 16, 1], 8)
    q, qf = lh.query(rng, 4)
    acc = torch.zeros((4, HKV, bt.shape[1] * PS), device="cuda")
    out, _ = run_scored(c, bt, lens, q, acc, acc, 4)
    ws = ws_of(pkv.pkv_decode_workspace_bytes(4, bt.shape[1], 4))
    ref = torch.empty_like(out)
    pkv.pkv_decode_attention(c.pool, q, lh.dev(bt), bt.shape[1], lh.dev(lens), 4, lh.SCALE, 4, ws, ws.numel(), ref)
    if kv == "bf16":
        assert torch.equal(out, ref)
    for b, L in enumerate(lens):
        off = lh.attend(qf[b], *c.rows(bt[b], range(int(L))), kv)[1]
        close(out[b], lh.bf16_values(ref[b]), 2 * off, b)
    c.close()


def test_scored_fp8_weights_see_small_query_entries():
    """Query entries 2^-11 to 2^-14 of their row's largest, which meets keys of nothing: the scores are
    the small entries' alone, and as exact as FP32 sums of their products."""
    rng = np.random.default_rng(77)
    c, bt, lens, _ = whole_case("fp8", [200, 33], 53)
    P = c.f8
    for b, L in enumerate(lens):
        t = np.arange(int(L))
        codes = P.index[bt[b][t // PS], 0, :, t % PS]                 # [L][8][64] of K
        k = rng.integers(0x30, 0x58, codes.shape).astype(np.uint8) | (rng.integers(0, 2, codes.shape) << 7).astype(np.uint8)
        k[..., 0] = 0
        c.host[codes] = k
        P.scales[bt[b][t // PS], 0, :, t % PS] = 2.0 ** 9             # keys of 2^8 to 2^13
    c.slab.copy_(torch.from_numpy(c.host).cuda())
    x = rng.uniform(1, 2, (2, HQ, D)) * 2.0 ** -rng.integers(12, 15, (2, HQ, D)) * rng.choice([-1, 1], (2, HQ, D))
    x[..., 0] = 1.0
    bits = lh.bf16_bits(x)
    q = torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16)
    qf, q = q.double().numpy(), q.cuda()
    acc = torch.zeros((2, HKV, bt.shape[1] * PS), device="cuda")
    run_scored(c, bt, lens, q, acc, acc)
    got = acc.cpu().numpy().astype(np.float64)
    for b, L in enumerate(lens):
        K, _ = c.rows(bt[b], range(int(L)))
        p, s = lh.weights(qf[b], K)
        ds = lh.SCALE * 2.0 ** -18 * np.einsum("hd,hnd->hn", np.abs(qf[b]), np.abs(np.repeat(K, 4, 0))) + 2.0 ** -20 * (1 + np.abs(s))
        assert np.ptp(s, axis=1).min() > 1 and ds.max() < 2.0 ** -9  # (an entry's last two bits move scores by more)
        dp = p * 2 * ds.max(1, keepdims=True) + 2.0 ** -126
        w, dw = p.reshape(HKV, 4, -1).sum(1), dp.reshape(HKV, 4, -1).sum(1)
        assert (np.abs(got[b, :, :L] - w) <= dw + 2.0 ** -22 * w).all(), b
    c.close()


@pytest.mark.parametrize("kv", KV)
def test_scored_device_checks(kv):
    c, bt, lens, rng = whole_case(kv, [100, 50, 40, 70], 12)
    q, _ = lh.query(rng, 4)
    bt2, lens2 = bt.copy(), lens.copy()
    bt2[0, 2], lens2[1], lens2[3] = -1, 0, bt.shape[1] * PS + 1
    acc = torch.full((4, HKV, bt.shape[1] * PS), 0.5, device="cuda")
    acc_out = torch.full_like(acc, -9.0)
    out, bits = run_scored(c, bt2, lens2, q, acc, acc_out, 128, ok=False)
    assert bits == pkv.PKV_DEVERR_LENGTH | pkv.PKV_DEVERR_PAGE_RANGE
    assert (acc_out[0, :, :100] == 0.5).all() and (acc_out[0, :, 100:] == -9.0).all()   # its only unit: no weight
    assert (acc_out[1] == -9.0).all() and (acc_out[3] == -9.0).all()
    total = (acc_out[2, :, :40] - 0.5).sum(-1)
    assert torch.allclose(total, torch.full_like(total, 4.0), atol=1e-4)   # 4 heads' weights, 40 roundings at 1
    assert not out[1].any() and not out[3].any()
    c.close()


# ------------------------------------------------------------------ evict

def plain_evict(acc, L, keep, recent, sinks):
    """The kept tokens of one (sequence, KV head), in order."""
    if L <= keep:
        return list(range(L))
    middle = range(sinks, L - recent)
    key = [-np.inf if np.isnan(acc[t]) else float(acc[t]) for t in middle]
    # NaN is below every number, minus infinity among them
    order = sorted(middle, key=lambda t: (np.isnan(acc[t]), -key[t - sinks], t))
    kept = set(range(sinks)) | set(range(L - recent, L)) | set(order[:keep - sinks - recent])
    return sorted(kept)


def run_evict(c, bt, lens, dst, acc, keep, recent, sinks, give_kept=True, in_place=False, ok=True):
    B, blocks = bt.shape
    dblocks = dst.shape[1]
    acc_d = lh.dev(acc)
    acc_out = acc_d if in_place else torch.full((B, HKV, dblocks * PS + 5), 3.0, device="cuda")
    kept = torch.full((B, HKV, keep), 77, dtype=torch.int32, device="cuda") if give_kept else None
    lens_d = lh.dev(lens)
    lens_out = lens_d if in_place else torch.full_like(lens_d, -9)
    nbytes = 0 if give_kept else pkv.pkv_evict_workspace_bytes(B, keep)
    ws, err = ws_of(nbytes), flag()
    pkv.pkv_evict(c.pool, lh.dev(bt), blocks, lens_d, B, lh.dev(dst), dblocks, keep, recent, sinks, acc_d, acc.shape[-1],
                  acc_out, acc_out.shape[-1], kept, lens_out, ws, nbytes, err)
    st, bits = pkv.pkv_check_device_error(err)
    if ok:
        assert (st, bits) == (pkv.PKV_OK, 0)
    return acc_out.cpu().numpy(), None if kept is None else kept.cpu().numpy(), lens_out.cpu().numpy(), bits


def acc_of(rng, shape, kind):
    if kind == "ties":                           # a handful of values, both zeros among them
        return rng.choice(np.array([0.0, -0.0, 0.5, 0.25, -1.0], np.float32), shape)
    if kind == "odd":
        x = rng.standard_normal(shape).astype(np.float32)
        x[rng.random(shape) < 0.2] = np.nan
        x[rng.random(shape) < 0.1] = np.inf
        x[rng.random(shape) < 0.1] = -np.inf
        x[rng.random(shape) < 0.1] = 1e-42       # subnormal
        return x
    if kind == "near":                           # neighbours of 1 between two far values
        x = (1 + rng.integers(0, 5000, shape) * 2.0 ** -23).astype(np.float32)
        x[rng.random(shape) < 0.001] = 3e38
        x[rng.random(shape) < 0.001] = -3e38
        return x
    return np.exp(2 * rng.standard_normal(shape)).astype(np.float32)


EVICTS = [
    # lengths, keep, recent, sinks, weights
    ([40], 8, 2, 1, "real"), ([40, 17, 8, 7, 1, 0], 8, 0, 0, "ties"), ([100, 33, 64], 32, 32, 0, "real"),
    ([100, 33, 64], 32, 20, 12, "odd"), ([200, 150], 1, 0, 0, "real"), ([200, 150, 1], 33, 1, 0, "odd"),
    ([1500, 1024, 1025, 2047], 700, 100, 4, "ties"), ([2600, 40], 1500, 0, 5, "real"), ([64, 65], 64, 10, 10, "odd"),
    ([300, 5], 299, 5, 5, "real"),
    # rows longer than the 8192 and 32768 weights that are held in registers
    ([9000, 8193, 20], 3000, 100, 4, "real"), ([33000, 32769], 5000, 500, 3, "ties"), ([16384], 4096, 0, 0, "odd"),
    ([40000, 33001], 6000, 100, 2, "real"),
    # crowded histograms: several steps over all weights
    ([3000, 700, 257], 600, 20, 3, "near"), ([20000], 7000, 0, 1, "near"), ([36000], 1000, 10, 0, "near"),
    # nothing up for choice; all but one
    ([5000, 70], 64, 60, 4, "real"), ([5000], 4999, 7, 2, "near"),
]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("case", range(len(EVICTS)))
def test_evict(kv, case):
    lens, keep, recent, sinks, kind = EVICTS[case]
    rng = np.random.default_rng(400 + case)
    lens = np.asarray(lens, dtype=np.int32)
    need, dneed = -(-lens // PS), -(-np.minimum(lens, keep) // PS)
    bt, n = lh.shuffled_tables(rng, need, int(need.max()) + 1)
    dst, m = lh.shuffled_tables(rng, dneed, int(dneed.max()), n)
    c = lh.Cache(kv, n + m)
    c.host[:] = rng.integers(0, 256, c.host.nbytes, dtype=np.uint8).view(c.host.dtype)   # any bytes move as they are
    c.upload()
    acc = acc_of(rng, (len(lens), HKV, bt.shape[1] * PS), kind)
    acc_out, kept, lens_out, _ = run_evict(c, bt, lens, dst, acc, keep, recent, sinks)
    got = c.download()
    want = c.host.copy()
    for b, L in enumerate(lens):
        nk = min(int(L), keep)
        assert lens_out[b] == nk
        for g in range(HKV):
            ids = plain_evict(acc[b, g], int(L), keep, recent, sinks)
            assert kept[b, g, :nk].tolist() == ids and (kept[b, g, nk:] == -1).all()
            assert np.array_equal(acc_out[b, g, :nk].view(np.uint32), acc[b, g, ids].view(np.uint32))
            assert (acc_out[b, g, nk:] == 0).all()
            src, ss = bt[b][np.array(ids, np.int64) // PS], np.array(ids, np.int64) % PS
            at = np.arange(nk)
            dp, ds = dst[b][at // PS], at % PS
            if kv == "bf16":
                P, W = ph.pool_view(c.host), ph.pool_view(want)
                W[dp, :, g, ds] = P[src, :, g, ss]
            else:
                P, W = ph.Fp8Pages(c.host), ph.Fp8Pages(want)
                W.pool[W.index[dp, :, g, ds]] = c.host[P.index[src, :, g, ss]]
                W.scales.view(np.uint32)[dp, :, g, ds] = P.scales.view(np.uint32)[src, :, g, ss]
    assert np.array_equal(got.view(np.uint8), want.view(np.uint8))       # nothing else has changed
    # the same without the list, and with weights and lengths in place
    c.slab.copy_(torch.from_numpy(c.host.view(np.uint8)).cuda())
    acc2, _, lens2, _ = run_evict(c, bt, lens, dst, acc, keep, recent, sinks, give_kept=False, in_place=True)
    assert np.array_equal(c.download().view(np.uint8), want.view(np.uint8)) and np.array_equal(lens2, lens_out)
    w = min(acc2.shape[-1], acc_out.shape[-1])
    assert np.array_equal(acc2[..., :w].view(np.uint32), acc_out[..., :w].view(np.uint32)) and (acc2[..., w:] == 0).all()
    c.close()


@pytest.mark.parametrize("kv", KV)
def test_evict_device_checks(kv):
    rng = np.random.default_rng(3)
    lens = np.array([100, 60, 97, 40], dtype=np.int32)
    bt, n = lh.shuffled_tables(rng, -(-lens // PS), 7)
    dst, m = lh.shuffled_tables(rng, np.array([2, 2, 2, 2]), 2, n)
    c = lh.Cache(kv, n + m).upload()
    start = c.download().copy()
    acc = acc_of(rng, (4, HKV, 7 * PS), "real")
    lens2, bt2, dst2 = lens.copy(), bt.copy(), dst.copy()
    lens2[0] = -1
    lens2[2] = 7 * PS + 1
    bt2[1, :], dst2[3, 1] = n + m, -4
    _, kept, lens_out, bits = run_evict(c, bt2, lens2, dst2, acc, 32, 4, 1, ok=False)
    assert bits == pkv.PKV_DEVERR_LENGTH | pkv.PKV_DEVERR_PAGE_RANGE
    assert lens_out.tolist() == [0, 32, 0, 32] and (kept[[0, 2]] == -1).all()
    got, page = c.download(), c.host.size // c.pages
    changed = {p for p in range(c.pages) if not np.array_equal(got[p * page:(p + 1) * page], start[p * page:(p + 1) * page])}
    assert changed <= {int(dst[3, 0])}           # sequence 1's sources and 3's second page are left out
    # destinations too short for what is kept
    _, kept, lens_out, bits = run_evict(c, bt, lens, dst, acc, 33, 4, 1, ok=False)
    assert bits == pkv.PKV_DEVERR_LENGTH and lens_out.tolist() == [0, 0, 0, 0]
    c.close()


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("with_q", [True, False])
def test_append_at(kv, with_q):
    rng = np.random.default_rng(17)
    B, blocks, max_pos = 7, 5, 4096
    pos = np.array([0, 4095, 77, 1, 2000, 16, 3000], dtype=np.int32)
    slots = np.array([0, 79, 15, 16, 33, 64, 5], dtype=np.int32)
    bt, n = lh.shuffled_tables(rng, np.full(B, blocks), blocks)
    c = lh.Cache(kv, n).upload()
    q, qf = lh.query(rng, B)
    kn, vn = rng.standard_normal((2, B, HKV, D))
    kn[3] = 0                                    # an all-zero row has scale 1
    kd, vd = (torch.from_numpy(lh.bf16_bits(x).view(np.int16).copy()).view(torch.bfloat16).cuda() for x in (kn, vn))
    rope, err = pkv.rope_table(max_pos, "cuda"), flag()
    out = torch.full_like(q, 7.0) if with_q else None
    pkv.pkv_append_rope_at(c.pool, kd, vd, q if with_q else None, out, lh.dev(bt), blocks, lh.dev(pos), lh.dev(slots), B,
                           rope, max_pos, err)
    assert pkv.pkv_check_device_error(err) == (pkv.PKV_OK, 0)
    got = c.download()
    want = lh.Cache(kv, n)                       # the same rows put where they belong
    for b in range(B):
        k = lh.rotated(kd[b].double().cpu().numpy(), pos[b])
        want.put(bt[b, slots[b] // PS], slots[b] % PS, k, vd[b].double().cpu().numpy())
        if with_q:
            close(out[b], lh.rotated(qf[b], pos[b]), 2.0 ** -8 * np.abs(lh.rotated(qf[b], pos[b])) + 2.0 ** -40)
        # K within one BF16 rounding (one E4M3 step on top for FP8 pages), V as it is
        gk, gv = c.rows(bt[b], [slots[b]], got)
        wk, wv = want.rows(bt[b], [slots[b]])
        assert np.array_equal(gv, wv)
        step = 2.0 ** -7 if kv == "bf16" else 2.0 ** -2
        assert (np.abs(gk - wk) <= step * np.abs(wk) + 2.0 ** -9 * np.abs(wk).max()).all()
        assert np.array_equal(gk, wk) or b not in (0, 3)
    mask = want.host.view(np.uint8) != lh.Cache(kv, n).host.view(np.uint8)
    assert np.array_equal(got.view(np.uint8)[~mask], c.host.view(np.uint8)[~mask]) or kv == "fp8"
    # the place its position: pkv_append_rope, bit for bit
    slots2 = np.minimum(pos, blocks * PS - 1).astype(np.int32)
    c.slab.copy_(torch.from_numpy(c.host.view(np.uint8)).cuda())
    q1 = q.clone()
    pkv.pkv_append_rope_at(c.pool, kd, vd, q, q1, lh.dev(bt), blocks, lh.dev(slots2), lh.dev(slots2), B, rope, max_pos, err)
    a = c.slab.clone()
    c.slab.copy_(torch.from_numpy(c.host.view(np.uint8)).cuda())
    q2 = q.clone()
    pkv.pkv_append_rope(c.pool, kd, vd, q2, lh.dev(bt), blocks, lh.dev(slots2), B, rope, max_pos, err)
    assert pkv.pkv_check_device_error(err) == (pkv.PKV_OK, 0)
    assert torch.equal(a, c.slab) and torch.equal(q1, q2)
    # device checks: the sequence is skipped
    start = c.slab.clone()
    bad = [(-1, 0), (max_pos, 0), (0, -1), (0, blocks * PS)]
    pkv.pkv_append_rope_at(c.pool, kd, vd, q, q1, lh.dev(bt), blocks, lh.dev(np.array([x[0] for x in bad], np.int32)),
                           lh.dev(np.array([x[1] for x in bad], np.int32)), 4, rope, max_pos, err)
    assert pkv.pkv_check_device_error(err) == (pkv.PKV_ERR_DEVICE_BOUNDS, pkv.PKV_DEVERR_LENGTH)
    assert torch.equal(start, c.slab) and torch.equal(q1, q2)
    c.close()


@pytest.mark.parametrize("max_pos", [4095, 20011])
def test_long_rope_tables(max_pos):
    """Filled by several threads: every row is there.  An angle p f of a frequency f <= 1, both
    rounded to 64 bits (the power to a unit in the last place), is p 2^-51 off at most between the
    two sides; the factors are held to 2^-48."""
    got = pkv.rope_table(max_pos, "cuda", lh.THETA).cpu().numpy().reshape(max_pos, D // 2, 4).astype(np.float64)
    p, i = np.arange(max_pos)[:, None], np.arange(D // 2)[None, :]
    angle = p * float(lh.THETA) ** (-2.0 * i / D)
    tol = max_pos * 2.0 ** -51 + 2.0 ** -47
    assert (np.abs(got[..., 0] + got[..., 2] - np.cos(angle)) <= tol).all()
    assert (np.abs(got[..., 1] + got[..., 3] - np.sin(angle)) <= tol).all()
