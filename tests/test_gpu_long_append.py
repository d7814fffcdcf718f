"""What an append leaves alone: every byte of the pool that is not one of its rows'."""
import numpy as np
import pytest
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import long_helpers as lh
from tests import paged_helpers as ph
from tests import test_gpu_long as tl
from tests import test_gpu_long_engine as te

pytestmark = pytest.mark.gpu

native = tl.native


def rows_mask(c, pages, slots):
    """The bytes of the rows at (page, slot): codes and scales of both, all heads."""
    mask = np.zeros_like(c.host)
    if c.kv == "bf16":
        ph.pool_view(mask)[pages, :, :, slots] = 0xFFFF
    else:
        f8 = ph.Fp8Pages(mask)
        mask[f8.index[pages, :, :, slots]] = 0xFF
        f8.scales.view(np.uint32)[pages, :, :, slots] = 0xFFFFFFFF
    return mask.view(np.uint8) != 0


@pytest.mark.parametrize("kv", tl.KV)
@pytest.mark.parametrize("call", ["append_at", "append", "step_window"])
def test_nothing_but_the_new_rows_changes(kv, call):
    rng = np.random.default_rng(19)
    B, blocks, max_pos = 18, 3, 64
    slots = np.concatenate([np.arange(16) + 16, [0, 47]]).astype(np.int32)   # every slot of a page
    bt, n = lh.shuffled_tables(rng, np.full(B, blocks), blocks)
    c = lh.Cache(kv, n + 2)
    c.host[:] = rng.integers(0, 256, c.host.nbytes, dtype=np.uint8).view(c.host.dtype)
    c.upload()
    q = te.bf16_dev(rng, (B, lh.HQ, lh.D))
    kn, vn = te.bf16_dev(rng, (B, lh.HKV, lh.D)), te.bf16_dev(rng, (B, lh.HKV, lh.D))
    rope, err, bt_d, at = pkv.rope_table(max_pos, "cuda"), tl.flag(), lh.dev(bt), lh.dev(slots)
    if call == "append_at":
        pkv.pkv_append_rope_at(c.pool, kn, vn, q, q, bt_d, blocks, 63 - at, at, B, rope, max_pos, err)
    elif call == "append":
        pkv.pkv_append_rope(c.pool, kn, vn, q, bt_d, blocks, at, B, rope, max_pos, err)
    else:
        nbytes = pkv.pkv_decode_window_workspace_bytes(B, blocks, 20, 2, 1)
        pkv.pkv_decode_step_window(c.pool, kn, vn, q, bt_d, blocks, at + 1, B, rope, max_pos, lh.SCALE, 20, 2, 1,
                                   tl.ws_of(nbytes), nbytes, torch.empty_like(q), err)
    assert pkv.pkv_check_device_error(err) == (pkv.PKV_OK, 0)
    mask = rows_mask(c, bt[np.arange(B), slots // lh.PS], slots % lh.PS)
    row = lh.HKV * (lh.D * 2 if kv == "bf16" else lh.D + 4)
    assert mask.sum() == B * 2 * row
    got, was = c.download().view(np.uint8), c.host.view(np.uint8)
    assert np.array_equal(got[~mask], was[~mask])
    assert (got[mask] != was[mask]).mean() > 0.9   # random bytes: one in 256 is what it was
    c.close()
