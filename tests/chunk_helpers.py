"""Test-side helpers for the attention of chunks: sequences with their pages, plain attention in 64 bits
and what the kernels may be off by."""
import numpy as np
import torch

from paged_kv_decode_12_gb300 import pkv
from tests import long_helpers as lh

PS, HKV, HQ, D, GROUP = lh.PS, lh.HKV, lh.HQ, lh.D, lh.GROUP
SENTINEL = 7.0


def seen(p, window, sinks):
    """Tokens that the token at position p attends to."""
    if not window:
        return np.arange(p + 1)
    lo = max(0, p + 1 - window)
    return np.concatenate([np.arange(min(sinks, lo)), np.arange(lo, p + 1)])


def attend(q, K, V, kv):
    """lh.attend for one token's rows with weights rounded to BF16 on either kind of pages, and
    a sum that is of the rounded weights: its rounding (2^-8) takes another |out| 2^-8."""
    out, off, _, _ = lh.attend(q, K, V, kv, rounding=2.0 ** -8)
    return out, off + 2.0 ** -8 * np.abs(out)


class Batch:
    """Sequences (cached, new) with rows for every token that a new one attends to; other places are
    NaN and pages without such a token are -1 in the table."""

    def __init__(self, kv, sizes, window=0, sinks=0, seed=0, blocks=None, spare=0, pad=0):
        self.rng = rng = np.random.default_rng(seed)
        self.kv, self.sizes, self.window, self.sinks = kv, sizes, window, sinks
        new = np.array([n for _, n in sizes])
        self.lens = np.array([c + n for c, n in sizes], np.int32)
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = max(1, int(new.sum()) + pad)
        need = -(-self.lens // PS)
        self.blocks = blocks or max(1, int(need.max()))
        self.tokens = [np.unique(np.concatenate([seen(p, window, sinks) for p in range(c, c + n)] or [[]])).astype(int)
                       for c, n in sizes]
        live = [sorted({int(t) // PS for t in tokens}) for tokens in self.tokens]
        ids = rng.permutation(sum(map(len, live)) + spare)
        self.bt = np.full((len(sizes), self.blocks), -1, np.int32)
        at = 0
        for b, pages in enumerate(live):
            self.bt[b, pages] = ids[at:at + len(pages)]
            at += len(pages)
        self.cache = lh.Cache(kv, max(1, at + spare))
        for b in range(len(sizes)):
            lh.fill(self.cache, self.bt[b], self.tokens[b], rng)
        self.q, self.qf = lh.query(rng, self.T)

    def upload(self):
        self.cache.upload()
        self.nbytes = pkv.pkv_chunk_attention_workspace_bytes(len(self.sizes), self.T)
        self.ws = torch.zeros(self.nbytes, dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = torch.full((self.T, HQ, D), SENTINEL, dtype=torch.bfloat16, device="cuda")
        self.dev = {x: lh.dev(getattr(self, x)) for x in ("bt", "lens", "starts")}
        return self

    def call(self, stream=None, options=0, **change):
        a = dict(self.dev, q=self.q, out=self.out, ws=self.ws, scale=lh.SCALE)
        a.update(change)
        pkv.pkv_chunk_attention(self.cache.pool, a["q"], a["bt"], self.blocks, a["lens"], a["starts"], len(self.sizes), self.T,
                                a["scale"], self.window, self.sinks, a["ws"], self.nbytes, a["out"], self.err, stream, options)
        return self

    def flag(self):
        torch.cuda.synchronize()
        return int(self.err)

    def check(self, rows=None, out=None):
        """The outputs of the sequences ``rows`` (all), and the rows behind the last left alone."""
        got = lh.bf16_values(self.out if out is None else out)
        for b in range(len(self.sizes)) if rows is None else rows:
            c, n = self.sizes[b]
            if not n:
                continue
            K, V = self.cache.rows(self.bt[b], self.tokens[b])
            for i in range(n):
                t = self.starts[b] + i
                pick = np.searchsorted(self.tokens[b], seen(c + i, self.window, self.sinks))
                want, off = attend(self.qf[t], K[:, pick], V[:, pick], self.kv)
                bad = ~(np.abs(got[t] - want) <= off)
                assert not bad.any(), ((b, i), np.argwhere(bad)[:4].tolist(), got[t][bad][:4], want[bad][:4], off[bad][:4])
        if rows is None:
            assert (got[self.starts[-1]:] == SENTINEL).all()
        return self

    def close(self):
        self.cache.close()
