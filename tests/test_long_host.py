"""CPU-only checks of the long-context entry points: workspace sizes and the refusals made before
any CUDA call."""
import numpy as np
import pytest

from paged_kv_decode_12_gb300 import pkv

A = 0x7F0000000000  # an aligned address, never dereferenced by host code
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_12_gb300 import _build

    _build.build()


@pytest.fixture(params=["bf16", "fp8"])
def pool(request):
    make = pkv.pkv_pool_create if request.param == "bf16" else pkv.pkv_pool_create_fp8
    p = make(A, 8 * pkv.PKV_PAGE_BYTES)
    yield p
    pkv.pkv_pool_destroy(p)


WINDOW = dict(q=A, bt=A, max_blocks=128, lens=A, B=4, scale=0.125, window=100, sinks=4, ppc=0, ws=A, nbytes=BIG, out=A,
              err=None, stream=0, options=0)
STEP = dict(k=A, v=A, q=A, bt=A, max_blocks=128, lens=A, B=4, rope=A, max_pos=2048, scale=0.125, window=100, sinks=4,
            ppc=0, ws=A, nbytes=BIG, out=A, err=None, stream=0, options=0)
SHARED = dict(q=A, bt=A, max_blocks=128, lens=A, B=4, starts=A, prefix=A, groups=2, max_prefix=64, scale=0.125, ppc=0,
              prefix_ppc=0, ws=A, nbytes=BIG, out=A, err=None, stream=0, options=0)
SCORED = dict(q=A, bt=A, max_blocks=128, lens=A, B=4, scale=0.125, acc=A, acc_out=A, stride=2048, ppc=0, ws=A,
              nbytes=BIG, out=A, err=None, stream=0, options=0)
EVICT = dict(bt=A, src_blocks=128, lens=A, B=4, dst=A, dst_blocks=32, keep=512, recent=64, sinks=4, acc=A, stride=2048,
             acc_out=A + 65536, out_stride=512, kept=None, lens_out=A, ws=A, nbytes=BIG, err=None, stream=0)
APPEND = dict(k=A, v=A, q=A, q_out=A, bt=A, max_blocks=128, pos=A, slots=A, B=4, rope=A, max_pos=2048, err=None, stream=0)

ATTENTION = [dict(q=None), dict(bt=None), dict(lens=None), dict(out=None), dict(q=A + 8), dict(out=A + 2), dict(ws=A + 4),
             dict(B=0), dict(B=-1), dict(B=65536), dict(max_blocks=0), dict(max_blocks=(1 << 20) + 1), dict(ppc=-1),
             dict(ppc=129), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
             dict(ws=None), dict(options=9), dict(options=0x400), dict(options=pkv.PKV_STEP_RING(1)),
             dict(options=pkv.PKV_DECODE_SPLIT_MERGE)]
CASES = [(pkv.pkv_decode_window, WINDOW, c) for c in ATTENTION + [dict(window=0), dict(window=-5), dict(sinks=-1)]]
CASES += [(pkv.pkv_decode_step_window, STEP, c) for c in ATTENTION + [dict(window=0), dict(sinks=-1), dict(k=None),
                                                                      dict(v=None), dict(rope=None), dict(max_pos=0)]]
CASES += [(pkv.pkv_decode_shared, SHARED, c) for c in ATTENTION + [dict(starts=None), dict(prefix=None), dict(groups=0),
                                                                   dict(groups=5), dict(max_prefix=-1),
                                                                   dict(max_prefix=129), dict(prefix_ppc=-1)]]
CASES += [(pkv.pkv_decode_scored, SCORED, c) for c in ATTENTION + [dict(acc=None), dict(acc_out=None), dict(stride=2047),
                                                                   dict(acc=A + 2), dict(acc_out=A + 1)]]
CASES += [(pkv.pkv_evict, EVICT, c) for c in [
    dict(bt=None), dict(lens=None), dict(dst=None), dict(acc=None), dict(acc_out=None), dict(lens_out=None), dict(B=0),
    dict(B=65536), dict(keep=0), dict(keep=67), dict(recent=-1), dict(sinks=-1), dict(recent=509), dict(src_blocks=0),
    dict(dst_blocks=0), dict(stride=2047), dict(out_stride=511), dict(acc=A + 1), dict(acc_out=A + 2), dict(ws=None),
    dict(ws=A + 2), dict(acc=A + 64, acc_out=A + 64, out_stride=4096)]]
CASES += [(pkv.pkv_append_rope_at, APPEND, c) for c in [
    dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(bt=None), dict(pos=None), dict(slots=None),
    dict(rope=None), dict(B=0), dict(max_blocks=0), dict(max_pos=0), dict(k=A + 8), dict(q_out=A + 4)]]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_refused_before_any_cuda_call(pool, case):
    fn, args, change = CASES[case]
    if fn is pkv.pkv_evict and "recent" not in change and "sinks" not in change and change.get("keep") == 67:
        assert args["recent"] + args["sinks"] > 67
    with pytest.raises(pkv.PkvError) as e:
        fn(pool, *dict(args, **change).values())
    assert e.value.status == pkv.PKV_ERR_INVALID_ARG, (fn.__name__, change)


@pytest.mark.parametrize("fn,args", [(pkv.pkv_decode_window, WINDOW), (pkv.pkv_decode_step_window, STEP),
                                     (pkv.pkv_decode_shared, SHARED), (pkv.pkv_decode_scored, SCORED)])
def test_workspace_and_policies(pool, fn, args):
    with pytest.raises(pkv.PkvError) as e:
        fn(pool, *dict(args, nbytes=64).values())
    assert e.value.status == pkv.PKV_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(pkv.PkvError) as e:
        fn(pool, *dict(args, options=pkv.PKV_DECODE_SIMT).values())
    assert e.value.status == pkv.PKV_ERR_UNSUPPORTED


def test_shared_has_no_sorted_order(pool):
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_decode_shared(pool, *dict(SHARED, options=pkv.PKV_STEP_SORTED).values())
    assert e.value.status == pkv.PKV_ERR_UNSUPPORTED


def test_null_pool():
    for fn, args in ((pkv.pkv_decode_window, WINDOW), (pkv.pkv_decode_step_window, STEP), (pkv.pkv_decode_shared, SHARED),
                     (pkv.pkv_decode_scored, SCORED), (pkv.pkv_evict, EVICT), (pkv.pkv_append_rope_at, APPEND)):
        with pytest.raises(pkv.PkvError) as e:
            fn(None, *args.values())
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG


def test_evict_workspace_is_the_kept_list(pool):
    assert pkv.pkv_evict_workspace_bytes(3, 100) == 3 * 8 * 100 * 4
    assert pkv.pkv_evict_workspace_bytes(0, 100) == 0 and pkv.pkv_evict_workspace_bytes(3, 0) == 0
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_evict(pool, *dict(EVICT, nbytes=4 * 8 * 512 * 4 - 1).values())
    assert e.value.status == pkv.PKV_ERR_WORKSPACE_TOO_SMALL


def test_workspace_bytes():
    # a window's workspace goes by the pages a sequence can visit, not by the table
    small = pkv.pkv_decode_window_workspace_bytes(4, 1 << 16, 100, 4, 4)
    assert small == pkv.pkv_decode_workspace_bytes(4, 1 + 8, 4)          # 1 page of sinks, at most 8 of 100 tokens
    assert pkv.pkv_decode_window_workspace_bytes(4, 5, 100, 4, 4) == pkv.pkv_decode_workspace_bytes(4, 5, 4)
    assert pkv.pkv_decode_window_workspace_bytes(4, 128, 2**31 - 1, 2**31 - 1, 16) == \
        pkv.pkv_decode_workspace_bytes(4, 128, 16)
    assert pkv.pkv_decode_window_workspace_bytes(4, 128, 0, 0, 16) == 0
    assert pkv.pkv_decode_shared_workspace_bytes(4, 128, 5, 0, 0, 0) == 0
    # 128 bytes of scores per table token, and one sum per query head
    a = pkv.pkv_decode_workspace_bytes(4, 128, 16)
    n = (a + 255) // 256 * 256 + 4 * 128 * 16 * 128 + 512
    assert pkv.pkv_decode_scored_workspace_bytes(4, 128, 16) == n
    assert pkv.pkv_decode_scored_workspace_bytes(4, 0, 16) == 0


def test_window_pages_bound():
    # n tokens in a row, whatever the first, touch at most (n + 14) // 16 + 1 pages
    for n in range(1, 100):
        most = max((s + n - 1) // 16 - s // 16 + 1 for s in range(16))
        assert most == (n + 14) // 16 + 1
        ws = pkv.pkv_decode_window_workspace_bytes(1, 1 << 20, n, 0, 1)
        assert ws == pkv.pkv_decode_workspace_bytes(1, most, 1), n
    assert np.iinfo(np.int32).max > 1 << 20
