"""Test-side helpers for the long-context operators: pools whose unused slots hold NaN, their
logical rows in 64 bits, and plain attention over any set of tokens."""
import numpy as np
import torch

import oracle
from paged_kv_decode_12_gb300 import pkv
from paged_kv_decode_12_gb300 import workloads as wl
from tests import paged_helpers as ph

HQ, HKV, D, PS = wl.NUM_Q_HEADS, wl.NUM_KV_HEADS, wl.HEAD_DIM, wl.PAGE_SIZE
GROUP = HQ // HKV
SCALE = 0.125
THETA = wl.ROPE_THETA

E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def bf16_bits(x: np.ndarray) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy() \
        .view(np.uint16)


def bf16_values(t: torch.Tensor) -> np.ndarray:
    return t.double().cpu().numpy()


class Cache:
    """A pool whose every slot is NaN until a row is put there, with an FP64 view of the rows."""

    def __init__(self, kv: str, pages: int):
        self.kv, self.pages = kv, pages
        if kv == "bf16":
            self.host = ph.new_pool(pages)
        else:
            self.host = np.full(pages * oracle.FP8_PAGE_BYTES, 0xFF, dtype=np.uint8)  # NaN codes and scales
            self.f8 = ph.Fp8Pages(self.host)
        self.slab = self.pool = None

    def put(self, page, slot, k, v):
        """Rows k, v [8][64] (float) at (page, slot)."""
        if self.kv == "bf16":
            P = ph.pool_view(self.host)
            P[page, 0, :, slot], P[page, 1, :, slot] = bf16_bits(k), bf16_bits(v)
            return
        for i, x in enumerate((k, v)):
            x = ph.bf16_to_f64(bf16_bits(x)).astype(np.float32)
            amax = np.abs(x).max(-1)
            scale = np.where(amax > 0, amax / np.float32(448), np.float32(1)).astype(np.float32)
            codes = torch.from_numpy(x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            for h in range(HKV):
                self.f8.set_row(page, i, h, slot, codes[h], scale[h])

    def upload(self):
        self.slab = torch.from_numpy(self.host.view(np.uint8).copy()).cuda()
        make = pkv.pkv_pool_create if self.kv == "bf16" else pkv.pkv_pool_create_fp8
        self.pool = make(self.slab, self.slab.numel())
        return self

    def download(self) -> np.ndarray:
        """The slab's bytes as they are on the device (of the host array's type)."""
        return self.slab.cpu().numpy().view(self.host.dtype)

    def rows(self, table_row, tokens, host=None):
        """K, V [8][n][64] in FP64 of the given tokens of one sequence."""
        host = self.host if host is None else host
        tokens = np.asarray(tokens, dtype=np.int64)
        pages, slots = np.asarray(table_row)[tokens // PS], tokens % PS
        if self.kv == "bf16":
            P = ph.pool_view(host)
            return tuple(ph.bf16_to_f64(P[pages, i, :, slots]).transpose(1, 0, 2) for i in (0, 1))
        f8 = ph.Fp8Pages(host)
        codes = E4M3[host[f8.index[pages, :, :, slots]]]                 # [n][2][8][64]
        x = codes * f8.scales[pages, :, :, slots].astype(np.float64)[..., None]
        return x[:, 0].transpose(1, 0, 2), x[:, 1].transpose(1, 0, 2)

    def close(self):
        if self.pool is not None:
            pkv.pkv_pool_destroy(self.pool)
            self.pool = None


def fill(cache, table_row, tokens, rng, outliers=0.02):
    """N(0, 1) rows at the given tokens; a few keys eight times as large."""
    for t in tokens:
        k, v = rng.standard_normal((2, HKV, D))
        if rng.random() < outliers:
            k = k * 8
        cache.put(table_row[t // PS], t % PS, k, v)


def weights(q, K):
    """Softmax weights [32][n] in FP64 of query rows [32][64] over keys [8][n][64], and the scores."""
    s = np.einsum("hd,hnd->hn", q, np.repeat(K, GROUP, 0)) * SCALE
    e = np.exp(s - s.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True), s


def attend(q, K, V, kv, rounding=None):
    """(output [32][64], what the kernels may be off by, weights, what those may be off by).

    The output is rounded once to BF16 (2^-8 relative).  The weights are rounded once for the
    second product: to BF16 (2^-8) or, on FP8 pages, to FP16 (2^-11) with a step of 2^-24 where
    they are small, in units of the largest V scale.  The scores are FP32 sums of 64 products
    (2^-18 of the products' absolute sum covers any order and a truncating adder); on FP8 pages a
    query entry below 2^-10 of its row's largest is off by at most 2^-17 of that largest.
    ``rounding``: the weights' rounding where a kernel has another than its pages' (a shared prefix
    of FP8 pages: BF16)."""
    p, s = weights(q, K)
    Kr, Vr = np.repeat(K, GROUP, 0), np.repeat(V, GROUP, 0)
    ds = SCALE * 2.0 ** -18 * np.einsum("hd,hnd->hn", np.abs(q), np.abs(Kr))
    if kv == "fp8":
        ds = ds + SCALE * 2.0 ** -17 * np.abs(q).max(-1)[:, None] * np.abs(Kr).sum(-1)
    ds = ds + 2.0 ** -20 * (1 + np.abs(s))
    dp = p * 2 * np.max(ds, axis=-1, keepdims=True) + 2.0 ** -126
    out = np.einsum("hn,hnd->hd", p, Vr)
    rounding = rounding or (2.0 ** -8 if kv == "bf16" else 2.0 ** -11)
    off = np.einsum("hn,hnd->hd", p * rounding + dp, np.abs(Vr))
    if kv == "fp8":
        off = off + 2.0 ** -24 * np.abs(Vr).max((1, 2))[:, None] * p.shape[1]
    return out, off + 2.0 ** -8 * np.abs(out) + 2.0 ** -126, p, dp


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def query(rng, B):
    bits = bf16_bits(rng.standard_normal((B, HQ, D)))
    t = torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def shuffled_tables(rng, need, blocks, first=0):
    """Tables [B][blocks] with need[b] distinct pages, -1 behind; and the number of pages."""
    ids = rng.permutation(int(np.sum(need))) + first
    bt = np.full((len(need), blocks), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    return bt, at


def rotated(x, pos):
    """x [..., 64] rotated to position pos, in FP64."""
    f = THETA ** (-2.0 * np.arange(D // 2) / D)
    w = np.exp(1j * pos * f)
    z = (x[..., :D // 2] + 1j * x[..., D // 2:]) * w
    return np.concatenate([z.real, z.imag], -1)
