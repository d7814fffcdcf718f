"""Attention of chunks whose outputs take the queries' place: an item's rows are written when every part of it has read
them."""
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import chunk_helpers as ch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


SIZES = [[(3000, 64)], [(3000, 1)], [(900, 20), (0, 200), (1500, 1)], [(i * 53 % 1200, 1 + (i % 7 == 0) * 40) for i in range(50)]]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_in_place(kv, case):
    b = ch.Batch(kv, SIZES[case], seed=301 + case, pad=case % 2).upload().call()
    assert b.flag() == 0
    given, rows = b.q.clone(), int(b.starts[-1])
    for _ in range(5):
        b.q.copy_(given)
        b.call(out=b.q)
        assert b.flag() == 0
        assert torch.equal(b.q[:rows], b.out[:rows])
        assert torch.equal(b.q[rows:], given[rows:])
    b.close()
