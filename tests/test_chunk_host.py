"""CPU-only checks of the entry points for chunks of new tokens: workspace sizes and the refusals made
before any CUDA call."""
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


TABLES = dict(lens=A, new=A, B=4, bt=A, max_blocks=128, layers=16, pages=A, num=100, used=A, used_out=A, max_tokens=64,
              starts=A, lens_out=A, pos=A, slots=A, ws=A, nbytes=BIG, err=None, stream=0)
APPEND = dict(k=A, k_stride=512, v=A, v_stride=512, q=A, q_stride=2048, q_out=A, q_norm=A, k_norm=A, eps=1e-5, slots=A,
              pos=A, pos_stride=7, axes=None, T=7, rope=A, max_pos=2048, err=None, stream=0)
ATTENTION = dict(q=A, bt=A, max_blocks=128, lens=A, starts=A, B=4, T=64, scale=0.125, window=0, sinks=0, ws=A, nbytes=BIG,
                 out=A, err=None, stream=0, options=0)

CASES = [(pkv.pkv_chunk_tables, TABLES, c) for c in [
    dict(lens=None), dict(new=None), dict(bt=None), dict(pages=None), dict(used=None), dict(used_out=None),
    dict(starts=None), dict(lens_out=None), dict(pos=None), dict(slots=None), dict(ws=None), dict(ws=A + 8),
    dict(slots=A + 4), dict(B=0), dict(B=4097), dict(max_blocks=0), dict(max_blocks=(1 << 20) + 1), dict(layers=0),
    dict(layers=65536), dict(num=-1), dict(max_tokens=0), dict(max_tokens=-5)]]
CASES += [(pkv.pkv_chunk_append, APPEND, c) for c in [
    dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(slots=None), dict(pos=None), dict(rope=None),
    dict(k_norm=None), dict(q_norm=None), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(k_stride=508), dict(v_stride=511), dict(q_stride=2044), dict(k_stride=514), dict(q_stride=2050),
    dict(q_stride=2052), dict(T=0), dict(T=-1), dict(T=1 << 30), dict(max_pos=0), dict(k=A + 4), dict(v=A + 2),
    dict(q=A + 4), dict(q_norm=A + 4), dict(slots=A + 4), dict(rope=A + 8), dict(axes=(8, 12, 11)),
    dict(axes=(8, 12, 13)), dict(axes=(-4, 18, 18)), dict(axes=(40, -4, -4)), dict(axes=(8, 12, 12), pos_stride=6)]]
CASES += [(pkv.pkv_chunk_attention, ATTENTION, c) for c in [
    dict(q=None), dict(bt=None), dict(lens=None), dict(starts=None), dict(out=None), dict(ws=None), dict(q=A + 8),
    dict(out=A + 2), dict(ws=A + 4), dict(B=0), dict(B=4097), dict(T=0), dict(T=1 << 30), dict(max_blocks=0),
    dict(max_blocks=(1 << 20) + 1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(window=-1), dict(sinks=-1), dict(sinks=4), dict(options=1), dict(options=0x400),
    dict(options=pkv.PKV_STEP_RING(2)), dict(options=pkv.PKV_STEP_SORTED)]]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_refused_before_any_cuda_call(pool, case):
    fn, args, change = CASES[case]
    with pytest.raises(pkv.PkvError) as e:
        fn(pool, *dict(args, **change).values())
    assert e.value.status == pkv.PKV_ERR_INVALID_ARG, (fn.__name__, change)


def test_axes_are_three():
    with pytest.raises(ValueError):
        pkv.pkv_chunk_append(None, *dict(APPEND, axes=(16, 16)).values())


def test_null_pool():
    for fn, args in ((pkv.pkv_chunk_tables, TABLES), (pkv.pkv_chunk_append, APPEND), (pkv.pkv_chunk_attention, ATTENTION)):
        with pytest.raises(pkv.PkvError) as e:
            fn(None, *args.values())
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG


def test_workspace_sizes(pool):
    for fn, args, size in ((pkv.pkv_chunk_tables, TABLES, pkv.pkv_chunk_tables_workspace_bytes(4)),
                           (pkv.pkv_chunk_attention, ATTENTION, pkv.pkv_chunk_attention_workspace_bytes(4, 64))):
        assert size > 0
        with pytest.raises(pkv.PkvError) as e:
            fn(pool, *dict(args, nbytes=size - 1).values())
        assert e.value.status == pkv.PKV_ERR_WORKSPACE_TOO_SMALL
    assert pkv.pkv_chunk_tables_workspace_bytes(0) == pkv.pkv_chunk_tables_workspace_bytes(4097) == 0
    for B, T in ((0, 5), (4097, 5), (4, 0), (4, 1 << 30)):
        assert pkv.pkv_chunk_attention_workspace_bytes(B, T) == 0
