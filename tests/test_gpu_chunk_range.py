"""Values far from 1: what an output may be off by besides rounding.

The tiles' weights lie between 2^-60 and 2 times the sum's least (BF16), so that their products with small values leave
what FP32 holds: a step of 16 tokens loses less than 2^-126, the sum is 2^-60 (1 - 2^-8) at least, which is below 2^-66 a
step and 2^-70 a token.  FP8 pages: row scales below 2^-100, of values below 448 2^-100 < 2^-91, count as 2^-100: less
than that."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import chunk_helpers as ch
from tests import long_helpers as lh

pytestmark = pytest.mark.gpu

PS, HKV, D = lh.PS, lh.HKV, lh.D


@pytest.fixture(scope="module", autouse=True)
def native():
    from paged_kv_decode_12_gb300 import _build

    _build.build()
    pkv.lib()


def filled(kv, sizes, size, apart=0.0, seed=0):
    """A batch whose values are ``size`` times a standard normal one (at most 4), and whose keys grow by ``apart`` a token."""
    b = ch.Batch(kv, sizes, seed=seed)
    for row, tokens in enumerate(b.tokens):
        for t in tokens:
            k, v = b.rng.standard_normal((2, HKV, D))
            b.cache.put(b.bt[row, t // PS], t % PS, k * (1 + t * apart), np.clip(v, -4, 4) * size)
    return b.upload()


def check(b, besides):
    got = lh.bf16_values(b.out)
    for row, (c, n) in enumerate(b.sizes):
        K, V = b.cache.rows(b.bt[row], b.tokens[row])
        for i in range(n):
            t, upto = b.starts[row] + i, c + i + 1
            want, off = ch.attend(b.qf[t], K[:, :upto], V[:, :upto], b.kv)
            bad = ~(np.abs(got[t] - want) <= off + besides * upto)
            assert not bad.any(), ((row, i), got[t][bad][:4], want[bad][:4])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("log2", [37, 0, -40, -52, -62, -80, -100, -118])
def test_values_of_any_size(kv, log2):
    b = filled(kv, [(200, 40), (0, 70), (33, 2)], 2.0 ** log2, seed=(101 + log2) % 1000).call()
    assert b.flag() == 0
    check(b, 2.0 ** -70)
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("log2", [37, -40])
def test_with_scores_that_move_the_reference(kv, log2):
    b = filled(kv, [(300, 40), (0, 100)], 2.0 ** log2, apart=0.2, seed=151).call()
    assert b.flag() == 0
    check(b, 2.0 ** -70)
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("log2", [37, -62, -80, -100, -118])
def test_single_tokens_keep_small_values(kv, log2):
    """Weights of 1 for the largest score: what is left of 2^-126 a step of 16 tokens."""
    sizes = [(500, 1), (40, 1), (0, 1)]
    b = filled(kv, sizes, 2.0 ** log2, seed=171 + log2).call()
    assert b.flag() == 0
    check(b, 2.0 ** -126)
    b.close()
