"""CPU tests of who gives a page back: a scheduler's pages go through the scheduler alone."""
import numpy as np
import pytest

from paged_kv_decode_12_gb300 import pkv
from tests import test_sched_host as ts

built = ts.built


def refused(fn, *args):
    with pytest.raises(pkv.PkvError) as e:
        fn(*args)
    return e.value.status


def test_a_request_keeps_its_pages_until_it_ends():
    """A page given back behind the scheduler's back would be handed to a second request, and come back to the
    free list when the first one ends."""
    pool, s = ts.make(12, layers=2)
    pkv.pkv_sched_submit(s, 1, 40, 5)
    _, _, rows = pkv.pkv_sched_admit(s, 4, 2, 8)
    held = rows[rows >= 0]
    own = pkv.pkv_pool_alloc(pool, 2)
    assert held.size == 6 and pkv.pkv_pool_info(pool)["num_free"] == 4
    for ids in ([held[0]], held, [own[0], held[3]], [held[1], held[1]]):
        assert refused(pkv.pkv_pool_free, pool, ids) == pkv.PKV_ERR_INVALID_ARG
        assert refused(pkv.pkv_pool_check, pool, ids) == pkv.PKV_ERR_INVALID_ARG
        assert pkv.pkv_pool_info(pool)["num_free"] == 4
    pkv.pkv_pool_check(pool, own)                # nothing is freed by asking
    pkv.pkv_pool_check(pool, own)
    pkv.pkv_pool_free(pool, own)
    assert refused(pkv.pkv_pool_check, pool, own) == pkv.PKV_ERR_DOUBLE_FREE
    assert refused(pkv.pkv_pool_check, pool, [12]) == pkv.PKV_ERR_INVALID_ARG
    # a second request gets other pages, and the first one's come back once
    pkv.pkv_sched_submit(s, 2, 40, 2)
    _, _, more = pkv.pkv_sched_admit(s, 4, 2, 8)
    assert not set(more[more >= 0].tolist()) & set(held.tolist())
    pkv.pkv_sched_finish(s, 1)
    assert pkv.pkv_pool_info(pool)["num_free"] == 6
    pkv.pkv_sched_finish(s, 2)
    assert pkv.pkv_pool_info(pool)["num_free"] == 12
    again = pkv.pkv_pool_alloc(pool, 12)         # pages that a scheduler has given back are anybody's
    assert sorted(again.tolist()) == list(range(12))
    pkv.pkv_pool_free(pool, again)
    pkv.pkv_sched_destroy(s)
    pkv.pkv_pool_destroy(pool)


def test_pages_of_active_requests_come_back_with_the_scheduler():
    pool, s = ts.make(20, layers=2)
    for rid in (1, 2):
        pkv.pkv_sched_submit(s, rid, 30, 9)
    _, _, rows = pkv.pkv_sched_admit(s, 4, 2, 8)
    for _ in range(4):                           # crosses a page boundary
        pkv.pkv_sched_decode_batch(s, 4, 2, 8)
    assert pkv.pkv_pool_info(pool)["num_free"] == 20 - 2 * 2 * 3
    pkv.pkv_sched_destroy(s)
    assert pkv.pkv_pool_info(pool)["num_free"] == 20
    ids = pkv.pkv_pool_alloc(pool, 20)
    pkv.pkv_pool_free(pool, ids)
    assert np.unique(ids).size == 20
    pkv.pkv_pool_destroy(pool)


def test_check_refuses_null():
    assert refused(pkv.pkv_pool_check, None, [0]) == pkv.PKV_ERR_INVALID_ARG
