"""Evictions that leave room: the tokens that follow need no new tables."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from paged_kv_decode_12_gb300.engine import DecodeEngine
from tests import long_helpers as lh
from tests import test_gpu_long as tl
from tests import test_gpu_long_engine as te

pytestmark = pytest.mark.gpu

native = tl.native


@pytest.mark.parametrize("kv", tl.KV)
def test_tokens_after_an_eviction_with_room(kv):
    rng = np.random.default_rng(15)
    lens, blocks = np.array([70, 33, 0, 127], dtype=np.int32), 8
    B, keep, room = lens.size, 32, 20
    eng = DecodeEngine(60, 1, B, max_blocks=blocks, pages_per_chunk=3, max_pos=512, kv=kv)
    eng.build_tables(lens)
    for b in range(B):
        if lens[b]:
            pkv.pkv_prefill_append(eng.pool, *(te.bf16_dev(rng, (1, int(lens[b]), lh.HKV, lh.D)) for _ in range(2)),
                                   lh.dev(eng.bt_host[:, b]), blocks, 1, 0, int(lens[b]), eng.rope, eng.max_pos, eng.err)
    weights = tl.acc_of(rng, (B, lh.HKV, blocks * lh.PS), "real")
    acc = lh.dev(weights)
    ref = [te.rows_of(eng, kv, 0, b, range(int(lens[b]))) for b in range(B)]
    free = pkv.pkv_pool_info(eng.pool)["num_free"]
    with pytest.raises(ValueError):
        eng.evict(0, lens, acc, keep, 4, 1, room=-1)
    taken = pkv.pkv_pool_alloc(eng.pool, free - 31)
    with pytest.raises(pkv.PkvError) as e:
        eng.evict(0, lens, acc, 128, 4, 1, room=10 ** 9)     # whole rows of pages, 32: more than the pool has left
    assert e.value.status == pkv.PKV_ERR_OUT_OF_PAGES
    pkv.pkv_pool_free(eng.pool, taken)
    assert pkv.pkv_pool_info(eng.pool)["num_free"] == free and np.array_equal(acc.cpu().numpy(), weights)
    slots = eng.evict(0, lens, acc, keep, 4, 1, room=room)
    assert slots.tolist() == [32, 32, 0, 32]
    assert (eng.bt_host >= 0).sum(-1).tolist() == [[4, 4, 2, 4]]      # 52 tokens, 52, 20, 52
    assert np.unique(eng.bt_host[eng.bt_host >= 0]).size == 14
    assert pkv.pkv_pool_info(eng.pool)["num_free"] == 60 - 14
    for b in range(B):
        ids = [tl.plain_evict(weights[b, g], int(lens[b]), keep, 4, 1) for g in range(lh.HKV)]
        ref[b] = tuple(np.stack([x[g, ids[g]] for g in range(lh.HKV)]) for x in ref[b])
    pos = lens.copy()
    for _ in range(room):
        q, kn, vn = te.bf16_dev(rng, (B, lh.HQ, lh.D)), te.bf16_dev(rng, (B, lh.HKV, lh.D)), te.bf16_dev(rng, (B, lh.HKV, lh.D))
        eng.append(0, kn, vn, q, lh.dev(pos), slots=lh.dev(slots))
        for b in range(B):
            new = te.rows_of(eng, kv, 0, b, [int(slots[b])])
            ref[b] = tuple(np.concatenate([x, y], 1) for x, y in zip(ref[b], new))
        pos, slots = pos + 1, slots + 1
        out = torch.empty_like(q)
        eng.attention(0, q, lh.dev(slots), out)
        qf = lh.bf16_values(q)
        for b in range(B):
            tl.close(out[b], *lh.attend(qf[b], *ref[b], kv)[:2], b)
    assert eng.check_errors() == (pkv.PKV_OK, 0)
    # room as far as the table is wide
    eng.evict(0, slots, acc, 10, 4, 1, room=100)
    assert (eng.bt_host >= 0).sum(-1).tolist() == [[7, 7, 7, 7]]
    eng.evict(0, np.full(B, 10), acc, 20, 4, 1, room=1000)
    assert (eng.bt_host >= 0).all() and eng.check_errors() == (pkv.PKV_OK, 0)
    eng.close()
