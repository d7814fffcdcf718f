"""Attention of chunks with starts that are no prefix sums: nothing is worked on, and every output row is zeros."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import chunk_helpers as ch
from tests import long_helpers as lh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


# sizes of sequences whose starts are then replaced; single tokens alone, among others, none
BAD = [
    ([(30, 5), (30, 4), (30, 11)], [[0, 5, 3, 20], [0, -4, 6, 20], [0, 5, 9, 21], [3, 5, 9, 20], [0, 12, 9, 20],
                                    [0, 5, 9, -1], [-(2 ** 31), 5, 9, 20], [0, 5, 9, 2 ** 31 - 1]]),
    ([(30, 1)], [[1, 1], [0, 2], [-1, 0], [1, 0]]),
    ([(30, 1), (200, 1), (7, 1)], [[0, 2, 1, 3], [1, 2, 3, 3], [0, 1, 2, 4], [0, 1, 0, 1]]),
    ([(30, 1)] * 40 + [(100, 60)], [[0] + [1, 0] * 20, list(range(1, 42)), list(range(40)) + [101]]),
]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("sizes,all_starts", BAD)
def test_all_outputs_are_zeros(kv, sizes, all_starts):
    b = ch.Batch(kv, sizes, seed=71).upload()
    good = b.dev["starts"].clone()
    for starts in all_starts:
        b.out.fill_(ch.SENTINEL)
        b.dev["starts"].copy_(lh.dev(np.array(starts + [starts[-1]] * (len(sizes) + 1 - len(starts)), np.int32)))
        b.call()
        assert b.flag() == pkv.PKV_DEVERR_LENGTH, starts
        assert not b.out.float().any(), starts
        b.err.zero_()
    # and the next call finds nothing changed
    b.dev["starts"].copy_(good)
    b.out.fill_(ch.SENTINEL)
    b.call()
    assert b.flag() == 0
    b.check().close()
