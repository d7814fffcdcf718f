"""The weights that scored attention gathers add up, however large the scores are."""
import numpy as np
import pytest
import torch

from tests import long_helpers as lh
from tests import test_gpu_long as tl

pytestmark = pytest.mark.gpu

native = tl.native


@pytest.mark.parametrize("kv", tl.KV)
@pytest.mark.parametrize("blocks", [20, 300])    # the weights added in the same launch, in a second one
@pytest.mark.parametrize("scale", [1, 64, 1024, 8192])
def test_weights_add_to_one(kv, blocks, scale):
    """Keys that are there several times, so that several tokens share the weight and the log of the sum is no
    whole number: a head's weights add to 1 whatever the largest score M is.  An entry is
    2^((x - M) - log2 l) with l the sum of 2^(x - M) as the kernel made it: it and l's terms are off by 2^-22
    each (the power) and by 2^-24 of their exponents, which tokens that weigh have small; the
    log by a unit in its last place (2^-20 below 16); l by 2^-24 for each of n additions and by
    2^-21 for each time it is rescaled, at most once a page, a warp and a chunk."""
    rng = np.random.default_rng(70 + scale)
    lens, copies = np.array([300, 112, 45, 16], dtype=np.int32), [3, 7, 5, 1]
    need = -(-lens // lh.PS)
    bt, n = lh.shuffled_tables(rng, need, blocks)
    c = lh.Cache(kv, n)
    for b, L in enumerate(lens):
        k = rng.standard_normal((int(L) // copies[b], lh.HKV, lh.D))
        for t in range(int(L)):
            c.put(bt[b, t // lh.PS], t % lh.PS, k[t % len(k)], rng.standard_normal((lh.HKV, lh.D)))
    c.upload()
    q, qf = lh.query(rng, lens.size)
    q, qf = q * scale, qf * scale                # a power of two: exact
    for ppc in (0, 2):
        acc = torch.zeros((lens.size, lh.HKV, blocks * lh.PS), device="cuda")
        out, _ = tl.run_scored(c, bt, lens, q, acc, acc, ppc)
        sums = acc.cpu().numpy().astype(np.float64).sum(-1)
        for b, L in enumerate(lens):
            K, V = c.rows(bt[b], range(int(L)))
            want, off, p, _ = lh.attend(qf[b], K, V, kv)
            tl.close(out[b], want, off, (b, L))
            assert scale < 1024 or np.abs(qf[b] @ K[0].T).max() * lh.SCALE > 1000
            tol = 3 * 2.0 ** -22 + 2.0 ** -20 + int(L) * 2.0 ** -24 + (need[b] + 16) * 2.0 ** -21
            assert (np.abs(sums[b] - 4) <= 4 * tol).all(), (ppc, b, sums[b] - 4, 4 * tol)
    c.close()
