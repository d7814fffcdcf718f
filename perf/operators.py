"""Decode operators for long contexts, as cases to be measured.

Five operators over the paged KV cache (32 query heads, 8 KV heads of 64 dims, 16-token pages,
BF16 pages or FP8 E4M3 pages with one scale per row), each for one new token per sequence:

``window``   attention over the last ``window`` tokens and the first ``sinks`` tokens
``shared``   attention of groups of sequences that share a prefix held once in the pool
``scored``   full attention that also adds every cached token's weight to an accumulator
``evict``    the cache cut to ``keep`` tokens per KV head by that accumulator
``append``   RoPE and append of a token whose position is not its cache slot

Where ``own`` is false ``run`` computes an operator with elementary torch operations in FP32;
where it is true it calls the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

HQ, HKV, GROUP, D, PAGE = 32, 8, 4, 64, 16
SCALE = 1.0 / math.sqrt(D)
THETA = 500000.0
BF16_PAGE = 2 * HKV * PAGE * D          # elements
UNIT = 2 * PAGE * (D + 4)               # bytes of one KV head of an FP8 page: codes, then row scales
CODES = 2 * PAGE * D
TOKEN_BYTES = {"bf16": 2 * HKV * D * 2, "fp8": 2 * HKV * (D + 4)}
MAX_POS = 65536                         # rows of the rotary table


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one chat session on its own, a short window: latency of a single small call
        dict(name="window_b1_w512", op="window", kv="bf16", batch=1, median=2048, longest=2048, window=512, sinks=4,
             ragged=1),
        # a serving batch with ragged histories; window and sinks that end inside pages
        dict(name="window_b64_w1000", op="window", kv="bf16", batch=64, median=1500, longest=8192, window=1000, sinks=5,
             ragged=2),
        # a large batch of long sessions over FP8 pages, most of whose pages have been given back
        dict(name="window_b256_w4096_fp8", op="window", kv="fp8", batch=256, median=12000, longest=32768, window=4096,
             sinks=16, ragged=3),
        # a few requests behind one short system prompt
        dict(name="shared_b4_p512", op="shared", kv="bf16", batch=4, groups=1, prefix=512, median=60, longest=256,
             ragged=4),
        # several prompts of different lengths with ragged groups, FP8 pages
        dict(name="shared_b72_g5_p6000_fp8", op="shared", kv="fp8", batch=72, groups=5, prefix=6000, median=300,
             longest=2048, ragged=5),
        # many questions about one long document
        dict(name="shared_b256_p32768", op="shared", kv="bf16", batch=256, groups=1, prefix=32768, median=100,
             longest=512, ragged=6),
        # one session that keeps score of its cache
        dict(name="scored_b1_l1024", op="scored", kv="bf16", batch=1, median=1024, longest=1024, ragged=7),
        # a ragged serving batch, FP8 pages
        dict(name="scored_b64_l16384_fp8", op="scored", kv="fp8", batch=64, median=4000, longest=16384, ragged=8),
        # one session's cache halved
        dict(name="evict_b1_k512", op="evict", kv="bf16", batch=1, median=1024, longest=1024, keep=512, recent=128,
             sinks=4, ragged=9),
        # a batch of long caches cut to a budget, FP8 pages
        dict(name="evict_b64_k2048_fp8", op="evict", kv="fp8", batch=64, median=6000, longest=8192, keep=2048,
             recent=500, sinks=4, ragged=10),
        # the append of one session after an eviction
        dict(name="append_b1", op="append", kv="bf16", batch=1, median=512, longest=512, ragged=11),
        # the append of a large batch, FP8 pages
        dict(name="append_b256_fp8", op="append", kv="fp8", batch=256, median=512, longest=2048, ragged=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_weight(c) for c in listed())
    while True:
        c = dict(op=rng.choice(["window", "shared", "scored", "evict", "append"]), kv=rng.choice(["bf16", "fp8"]),
                 ragged=rng.randrange(100, 1 << 30))
        if c["op"] == "window":
            c.update(batch=_log(rng, 1, 256), longest=_log(rng, 1, 32768), window=_log(rng, 1, 4096),
                     sinks=rng.choice([0, rng.randrange(0, 65)]))
            c["median"] = max(1, int(c["longest"] * rng.uniform(0.2, 1.0)))
        elif c["op"] == "shared":
            c.update(batch=_log(rng, 1, 256), prefix=_log(rng, 16, 32768), longest=_log(rng, 1, 2048))
            c["groups"] = _log(rng, 1, min(8, c["batch"]))
            c["median"] = max(1, int(c["longest"] * rng.uniform(0.2, 1.0)))
        elif c["op"] == "scored":
            c.update(batch=_log(rng, 1, 64), longest=_log(rng, 1, 16384))
            c["median"] = max(1, int(c["longest"] * rng.uniform(0.2, 1.0)))
        elif c["op"] == "evict":
            c.update(batch=_log(rng, 1, 64), longest=_log(rng, 16, 16384))
            c["median"] = max(1, int(c["longest"] * rng.uniform(0.4, 1.0)))
            c["keep"] = _log(rng, 8, 4096)
            c["recent"] = rng.randrange(0, c["keep"] + 1)
            c["sinks"] = rng.randrange(0, min(65, c["keep"] - c["recent"] + 1))
        else:
            c.update(batch=_log(rng, 1, 256), longest=_log(rng, 1, 2048))
            c["median"] = max(1, int(c["longest"] * rng.uniform(0.2, 1.0)))
        if _weight(c) <= most and _padded(c) <= 1 << 21:
            return c


def _lengths(case):
    """Ragged lengths of the case, drawn from its own seed (the same for every input): log-normal, the first the longest."""
    r = np.random.RandomState(case["ragged"])
    x = np.rint(r.lognormal(math.log(case["median"]), 0.6, case["batch"]))
    lens = np.clip(x, 1, case["longest"]).astype(np.int32)
    lens[0] = case["longest"]
    return lens


def _groups(case):
    """Row bounds of the groups and their prefix lengths in pages: ragged, the first the longest."""
    r = np.random.RandomState(case["ragged"] + 1)
    cuts = np.sort(r.choice(np.arange(1, case["batch"]), case["groups"] - 1, replace=False)) if case["groups"] > 1 else []
    starts = np.concatenate([[0], cuts, [case["batch"]]]).astype(np.int32)
    pages = (case["prefix"] * np.exp(-2.0 * r.rand(case["groups"])) / PAGE).astype(np.int32)
    pages[0] = case["prefix"] // PAGE
    return starts, pages


def _padded(case):
    """Tokens of the plain form's padded gathers (they bound its memory)."""
    n = case["batch"] * case["longest"]
    if case["op"] == "window":
        n = case["batch"] * (min(case["window"], case["longest"]) + case["sinks"])
    elif case["op"] == "shared":
        starts, pages = _groups(case)
        n += int(np.diff(starts).max()) * case["groups"] * int(pages.max()) * PAGE // 8 + case["groups"] * int(pages.max()) * PAGE
    return n


def _visible(case, lens):
    return np.minimum(lens, np.minimum(lens, case["window"]) + np.minimum(case["sinks"], np.maximum(lens - case["window"], 0)))


def work(case):
    lens = _lengths(case).astype(np.int64)
    B, per = case["batch"], TOKEN_BYTES[case["kv"]]
    io = B * HQ * D * 2 * 2                     # query rows in, output rows out
    if case["op"] == "window":
        n = int(_visible(case, lens).sum())
        return {"bytes": n * per + io, "flops": 4 * D * HQ * n}
    if case["op"] == "shared":
        starts, pages = _groups(case)
        pre = int(pages.sum()) * PAGE
        rows = int((np.diff(starts).astype(np.int64) * pages).sum()) * PAGE
        n = int(lens.sum())
        return {"bytes": (pre + n) * per + io, "flops": 4 * D * HQ * (rows + n)}
    if case["op"] == "scored":
        n = int(lens.sum())
        return {"bytes": n * per + io + n * HKV * 8, "flops": 4 * D * HQ * n}
    if case["op"] == "evict":
        kept = int(np.minimum(lens, case["keep"]).sum())
        return {"bytes": kept * per * 2 + int(lens.sum()) * HKV * 4 + kept * HKV * 8, "flops": 0}
    return {"bytes": B * (2 * HKV * D * 2 + per) + io + B * (D // 2) * 16, "flops": 6 * B * (HQ + HKV) * D // 2}


def _weight(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


# ------------------------------------------------------------------ FP8 pages

def _v_offsets(device):
    """Byte of the V code of (slot, dim) inside a KV head's V codes: slots 2p and 2p + 1 share a
    128-byte line of 16-byte chunks (8 dims of both), chunk c stored at c xor (2p mod 8)."""
    s = torch.arange(PAGE, device=device)[:, None]
    d = torch.arange(D, device=device)[None, :]
    p = s // 2
    return p * 2 * D + ((d // 8) ^ ((2 * p) % 8)) * 16 + (d % 8) * 2 + s % 2


def _quantize(x):
    """E4M3 codes (as bytes) and row scales of FP32 rows [..., 64]."""
    scale = x.abs().amax(-1) / 448.0
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _fill_pages(kv, pages, gen, device):
    """A slab of pages of N(0, 1) rows, one key row in a hundred eight times as large."""
    slab = torch.empty(pages * BF16_PAGE, dtype=torch.bfloat16, device=device) if kv == "bf16" else \
        torch.empty(pages * HKV * UNIT, dtype=torch.uint8, device=device)
    off = _v_offsets(device).reshape(-1)
    step = 8192
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = torch.randn((n, HKV, 2, PAGE, D), generator=gen, device=device)
        x[:, :, 0] *= torch.where(torch.rand((n, HKV, PAGE, 1), generator=gen, device=device) < 0.01, 8.0, 1.0)
        x = x.to(torch.bfloat16)
        if kv == "bf16":
            slab.view(pages, 2, HKV, PAGE, D)[at:at + n] = x.transpose(1, 2)
        else:
            codes, scale = _quantize(x.float())
            u = slab.view(pages, HKV, UNIT)[at:at + n]
            u[:, :, :PAGE * D] = codes[:, :, 0].reshape(n, HKV, PAGE * D)
            u[:, :, PAGE * D + off] = codes[:, :, 1].reshape(n, HKV, PAGE * D)
            u[:, :, CODES:] = scale.reshape(n, HKV, 2 * PAGE).view(torch.uint8)
    return slab


# ------------------------------------------------------------------ prepare

def _bf16(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _tables(need, blocks, r, first=0):
    """Block tables [B][blocks] with need[b] pages from a shuffled pool, -1 behind; and the page count."""
    total = int(need.sum())
    ids = (r.permutation(total) + first).astype(np.int32)
    bt = np.full((need.size, blocks), -1, dtype=np.int32)
    bt[np.arange(blocks)[None, :] < need[:, None]] = ids
    return bt, total


def prepare(case, seed):
    op, kv, B = case["op"], case["kv"], case["batch"]
    gen = torch.Generator("cuda").manual_seed(seed)
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    lens = _lengths(case)
    s = {"case": case, "kv": kv, "B": B}
    blocks = -(-int(lens.max()) // PAGE)
    need = -(-lens // PAGE)
    if op == "window":
        # pages that have slid out of the window have been given back: their entries are -1
        j = np.arange(blocks)[None, :]
        live = (j < need[:, None]) & ((j * PAGE < case["sinks"]) | ((j + 1) * PAGE > (lens - case["window"])[:, None]))
        pages = int(live.sum())
        bt = np.full((B, blocks), -1, dtype=np.int32)
        bt[live] = r.permutation(pages).astype(np.int32)
    elif op == "shared":
        starts, prefix = _groups(case)
        of_row = np.repeat(np.arange(case["groups"]), np.diff(starts))
        blocks = int((prefix[of_row] + need).max())
        pre, n0 = _tables(prefix, max(1, int(prefix.max())), r)
        tail, n1 = _tables(need, int(need.max()), r, n0)
        bt = np.full((B, blocks), -1, dtype=np.int32)
        j = np.arange(blocks)[None, :]
        shared = j < prefix[of_row][:, None]
        bt[shared] = pre[of_row][:, :blocks][j[:, :pre.shape[1]].repeat(B, 0) < prefix[of_row][:, None]]
        mine = (j >= prefix[of_row][:, None]) & (j < (prefix[of_row] + need)[:, None])
        bt[mine] = tail[tail >= 0]
        pages = n0 + n1
        lens = (lens + prefix[of_row] * PAGE).astype(np.int32)
        s.update(starts=torch.from_numpy(starts).cuda(), prefix=torch.from_numpy(prefix).cuda(), G=case["groups"],
                 max_prefix=int(prefix.max()))
        # rows of each group, padded with row 0, and each row's place
        n = np.diff(starts)
        at = np.minimum(starts[:-1, None] + np.arange(n.max())[None, :], B - 1)
        s.update(rows=torch.from_numpy(at.astype(np.int64)).cuda(), row_group=torch.from_numpy(of_row.astype(np.int64)).cuda(),
                 row_place=torch.from_numpy((np.arange(B) - starts[of_row]).astype(np.int64)).cuda(),
                 longest=int(need.max()) * PAGE)
    else:
        bt, pages = _tables(need, blocks, r)
    s.update(bt=torch.from_numpy(bt).cuda(), lens=torch.from_numpy(lens).cuda(), blocks=blocks, max_len=int(lens.max()),
             err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    spare = 0
    if op == "evict":
        dst_need = -(-np.minimum(lens, case["keep"]) // PAGE)
        dst, spare = _tables(dst_need, int(dst_need.max()), r, pages)
        s.update(dst=torch.from_numpy(dst).cuda(), dst_blocks=int(dst_need.max()), src_pages=pages)
    s["pages"] = pages + spare
    s["slab"] = _fill_pages(kv, s["pages"], gen, "cuda")
    if op in ("window", "shared", "scored", "append"):
        s["q"] = _bf16((B, HQ, D), gen)
        s["out"] = torch.empty_like(s["q"])
    if op in ("scored", "evict"):
        # weights gathered so far: a few tokens hold most of them, and many hold none at all; a
        # cache that is being scored has a few steps' worth of them
        acc = torch.exp(2.0 * torch.randn((B, HKV, blocks * PAGE), generator=gen, device="cuda"))
        acc = torch.where(torch.rand(acc.shape, generator=gen, device="cuda") < 0.2, torch.zeros_like(acc), acc)
        inside = torch.arange(blocks * PAGE, device="cuda") < s["lens"][:, None]
        if op == "scored":
            acc = acc * (GROUP / s["lens"].float())[:, None, None]
        s["acc"] = acc * inside[:, None, :]
        s["acc_out"] = torch.zeros_like(s["acc"]) if op == "scored" else \
            torch.zeros((B, HKV, s["dst_blocks"] * PAGE), device="cuda")
    if op == "evict":
        s["lens_out"] = torch.zeros_like(s["lens"])
        s["kept"] = torch.full((B, HKV, case["keep"]), -1, dtype=torch.int32, device="cuda")
    if op == "append":
        s["k_new"], s["v_new"] = _bf16((B, HKV, D), gen), _bf16((B, HKV, D), gen)
        s["slots"] = s["lens"] - 1
        s["pos"] = torch.randint(0, MAX_POS, (B,), generator=gen, device="cuda", dtype=torch.int32)
    if own:
        _own_handles(s)
    return s


def _own_handles(s):
    """The pool object, the workspace and the rotary table that a user's program keeps."""
    from paged_kv_decode_12_gb300 import pkv

    case, B, nbytes = s["case"], s["B"], s["slab"].numel() * s["slab"].element_size()
    s["pool"] = pkv.pkv_pool_create(s["slab"], nbytes) if s["kv"] == "bf16" else \
        pkv.pkv_pool_create_fp8(s["slab"], nbytes)
    ws = 0
    if case["op"] == "window":
        ws = pkv.pkv_decode_window_workspace_bytes(B, s["blocks"], case["window"], case["sinks"], 0)
    elif case["op"] == "shared":
        ws = pkv.pkv_decode_shared_workspace_bytes(B, s["blocks"], s["G"], s["max_prefix"], 0, 0)
    elif case["op"] == "scored":
        ws = pkv.pkv_decode_scored_workspace_bytes(B, s["blocks"], 0)
    elif case["op"] == "evict":
        ws = pkv.pkv_evict_workspace_bytes(B, case["keep"])
    else:
        s["rope"] = pkv.rope_table(MAX_POS, "cuda", THETA)
    s["ws"], s["ws_bytes"] = torch.zeros(max(ws, 16), dtype=torch.uint8, device="cuda"), ws


# ------------------------------------------------------------------ run

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from paged_kv_decode_12_gb300 import pkv

    case = s["case"]
    if case["op"] == "window":
        pkv.pkv_decode_window(s["pool"], s["q"], s["bt"], s["blocks"], s["lens"], s["B"], SCALE, case["window"],
                              case["sinks"], 0, s["ws"], s["ws_bytes"], s["out"], s["err"])
        return s["out"]
    if case["op"] == "shared":
        pkv.pkv_decode_shared(s["pool"], s["q"], s["bt"], s["blocks"], s["lens"], s["B"], s["starts"], s["prefix"],
                              s["G"], s["max_prefix"], SCALE, 0, 0, s["ws"], s["ws_bytes"], s["out"], s["err"])
        return s["out"]
    if case["op"] == "scored":
        pkv.pkv_decode_scored(s["pool"], s["q"], s["bt"], s["blocks"], s["lens"], s["B"], SCALE, s["acc"],
                              s["acc_out"], s["blocks"] * PAGE, 0, s["ws"], s["ws_bytes"], s["out"], s["err"])
        return {"out": s["out"], "acc": s["acc_out"]}
    if case["op"] == "evict":
        pkv.pkv_evict(s["pool"], s["bt"], s["blocks"], s["lens"], s["B"], s["dst"], s["dst_blocks"], case["keep"],
                      case["recent"], case["sinks"], s["acc"], s["blocks"] * PAGE, s["acc_out"],
                      s["dst_blocks"] * PAGE, s["kept"], s["lens_out"], s["ws"], s["ws_bytes"], s["err"])
        return _evicted(s, s["acc_out"], s["kept"], s["lens_out"])
    pkv.pkv_append_rope_at(s["pool"], s["k_new"], s["v_new"], s["q"], s["out"], s["bt"], s["blocks"], s["pos"],
                           s["slots"], s["B"], s["rope"], MAX_POS, s["err"])
    return _appended(s, s["out"])


def _pool_outputs(s, first):
    """The pages from `first` on as they stand, as the values they hold."""
    if s["kv"] == "bf16":
        return {"pages": s["slab"].view(-1, BF16_PAGE)[first:]}
    u = s["slab"].view(s["pages"], HKV, UNIT)[first:]
    return {"codes": u[:, :, :CODES].view(torch.float8_e4m3fn), "scales": u[:, :, CODES:].view(torch.float32)}


def _evicted(s, acc, kept, lens):
    return {"acc": acc, "kept": kept, "lens": lens, **_pool_outputs(s, s["src_pages"])}


def _appended(s, q):
    return {"q": q, **_pool_outputs(s, 0)}


def _gather(s, page, slot):
    """K and V rows [..., 8, 64] in FP32 at (page, slot)."""
    if s["kv"] == "bf16":
        x = s["slab"].view(s["pages"], 2, HKV, PAGE, D)
        return x[page, 0, :, slot].float(), x[page, 1, :, slot].float()
    u = s["slab"].view(s["pages"], HKV, UNIT)
    scales = u[:, :, CODES:].view(torch.float32).view(s["pages"], HKV, 2, PAGE)
    kc = u[:, :, :PAGE * D].view(s["pages"], HKV, PAGE, D)[page, :, slot]
    head = torch.arange(HKV, device=u.device)[:, None]
    off = _v_offsets(u.device)[slot][..., None, :] + PAGE * D
    vc = u[page[..., None, None], head, off]
    return (kc.view(torch.float8_e4m3fn).float() * scales[page, :, 0, slot][..., None],
            vc.view(torch.float8_e4m3fn).float() * scales[page, :, 1, slot][..., None])


def _tokens(s, t, valid):
    """K and V [B, n, 8, 64] of tokens t [B, n] of every sequence (anything where not valid)."""
    t = torch.where(valid, t, torch.zeros_like(t))
    page = torch.gather(s["bt"], 1, t // PAGE).long()
    page = torch.where(valid, page, torch.zeros_like(page))
    return _gather(s, page, t % PAGE)


def _attend(q, k, v, valid):
    """Softmax attention of q [B, 32, 64] over k, v [B, n, 8, 64]; the output and the weights."""
    qg = q.float().view(-1, HKV, GROUP, D)
    x = torch.einsum("bghd,bngd->bghn", qg, k) * SCALE
    x = x.masked_fill(~valid[:, None, None, :], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    return torch.einsum("bghn,bngd->bghd", p, v).reshape(-1, HQ, D).to(torch.bfloat16), p


def _run_plain(s):
    return {"window": _plain_window, "shared": _plain_shared, "scored": _plain_scored, "evict": _plain_evict,
            "append": _plain_append}[s["case"]["op"]](s)


def _plain_window(s):
    W, S = min(s["case"]["window"], s["max_len"]), min(s["case"]["sinks"], s["max_len"])
    L = s["lens"].long()[:, None]
    head = torch.arange(S, device="cuda")[None, :].expand(s["B"], S)
    tail = L - W + torch.arange(W, device="cuda")[None, :]
    t = torch.cat([head, tail], 1)
    valid = torch.cat([head < L - W, tail >= 0], 1)
    k, v = _tokens(s, t, valid)
    return _attend(s["q"], k, v, valid)[0]


def _plain_shared(s):
    G, P = s["G"], s["max_prefix"] * PAGE
    pre = s["prefix"].long()
    q = s["q"].float().view(-1, HKV, GROUP, D)
    # the rows' own tokens
    n = s["longest"]
    t = pre[s["row_group"]][:, None] * PAGE + torch.arange(n, device="cuda")[None, :]
    valid = t < s["lens"][:, None]
    k, v = _tokens(s, t, valid)
    x = torch.einsum("bghd,bngd->bghn", q, k) * SCALE
    x = x.masked_fill(~valid[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    if P:
        # the prefix, once for each group: its rows side by side, padded to the largest group
        t = torch.arange(P, device="cuda")[None, :].expand(G, P)
        inside = t < pre[:, None] * PAGE
        page = torch.gather(s["bt"][s["starts"][:-1].long()], 1, t // PAGE).long()
        kp, vp = _gather(s, torch.where(inside, page, torch.zeros_like(page)), t % PAGE)
        qp = q[s["rows"]]                                                     # [G, n, 8, 4, 64]
        xp = torch.einsum("rnghd,rpgd->rgnhp", qp, kp) * SCALE
        xp = xp.masked_fill(~inside[:, None, None, None, :], -math.inf)
        mp = xp.amax(-1)                                                       # [G, 8, n, 4]
        mr = torch.maximum(m, mp[s["row_group"], :, s["row_place"]][..., None])
        ep = torch.exp(xp - mr[..., 0][s["rows"]].transpose(1, 2)[..., None])
        lp = ep.sum(-1)[s["row_group"], :, s["row_place"]]
        op = torch.einsum("rgnhp,rpgd->rgnhd", ep, vp)[s["row_group"], :, s["row_place"]]
        m = mr
    e = torch.exp(x - m)
    l, o = e.sum(-1), torch.einsum("bghn,bngd->bghd", e, v)
    if P:
        l, o = l + lp, o + op
    return (o / l[..., None]).reshape(-1, HQ, D).to(torch.bfloat16)


def _plain_scored(s):
    n = s["blocks"] * PAGE
    t = torch.arange(n, device="cuda")[None, :].expand(s["B"], n)
    valid = t < s["lens"][:, None]
    k, v = _tokens(s, t, valid)
    out, p = _attend(s["q"], k, v, valid)
    return {"out": out, "acc": s["acc"] + p.sum(2)}


def _plain_evict(s):
    case, B = s["case"], s["B"]
    keep, recent, sinks = case["keep"], case["recent"], case["sinks"]
    L = s["lens"].long()[:, None, None]
    n = s["acc"].shape[-1]
    t = torch.arange(n, device="cuda")
    must = (t < sinks) | (t >= L - recent) | (L <= keep)
    key = torch.where(must, math.inf, s["acc"])
    key = torch.where((t < L).expand_as(key), key, -math.inf)
    # the largest first, of equal ones the lowest index; then the kept ones in their own order
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    count = L.clamp(max=keep)
    place = torch.arange(order.shape[-1], device="cuda")
    order = torch.where(place < count, order, n)
    order = torch.sort(order, dim=-1).values
    valid = place < count
    got = torch.where(valid, order, 0)
    kept = torch.full((B, HKV, keep), -1, dtype=torch.int32, device="cuda")
    kept[..., :order.shape[-1]] = torch.where(valid, order, -1).int()
    acc = torch.zeros_like(s["acc_out"])
    w = min(acc.shape[-1], order.shape[-1])
    acc[..., :w] = torch.where(valid, torch.gather(s["acc"], 2, got), 0.0)[..., :w]
    # every kept row's place in its new page
    src = torch.gather(s["bt"][:, None].expand(B, HKV, -1), 2, got // PAGE).long()
    b, g, i = torch.nonzero(valid.expand(B, HKV, -1), as_tuple=True)
    sp, ss = src[b, g, i], got[b, g, i] % PAGE
    dp, ds = s["dst"][b, i // PAGE].long(), i % PAGE
    if s["kv"] == "bf16":
        x = s["slab"].view(s["pages"], 2, HKV, PAGE, D)
        x[dp, :, g, ds] = x[sp, :, g, ss]
    else:
        u = s["slab"].view(s["pages"], HKV, UNIT)
        k = u[:, :, :PAGE * D].view(s["pages"], HKV, PAGE, D)
        k[dp, g, ds] = k[sp, g, ss]
        off = _v_offsets("cuda") + PAGE * D
        u[dp[:, None], g[:, None], off[ds]] = u[sp[:, None], g[:, None], off[ss]]
        scales = u[:, :, CODES:].view(torch.float32).view(s["pages"], HKV, 2, PAGE)
        scales[dp, g, :, ds] = scales[sp, g, :, ss]
    return _evicted(s, acc, kept, L[:, 0, 0].clamp(max=keep).int())


def _plain_append(s):
    i = torch.arange(D // 2, device="cuda", dtype=torch.float64)
    a = s["pos"].double()[:, None, None] * THETA ** (-2.0 * i / D)
    c, z = torch.cos(a), torch.sin(a)

    def turned(x):
        x1, x2 = x.double()[..., :D // 2], x.double()[..., D // 2:]
        return torch.cat([x1 * c - x2 * z, x2 * c + x1 * z], -1).to(torch.bfloat16)

    q, k = turned(s["q"]), turned(s["k_new"])
    slot = s["slots"].long()
    page = torch.gather(s["bt"], 1, slot[:, None] // PAGE)[:, 0].long()
    if s["kv"] == "bf16":
        x = s["slab"].view(s["pages"], 2, HKV, PAGE, D)
        x[page, 0, :, slot % PAGE] = k
        x[page, 1, :, slot % PAGE] = s["v_new"]
        return _appended(s, q)
    u = s["slab"].view(s["pages"], HKV, UNIT)
    kc, ks = _quantize(k.float())
    vc, vs = _quantize(s["v_new"].float())
    u[:, :, :PAGE * D].view(s["pages"], HKV, PAGE, D)[page, :, slot % PAGE] = kc
    off = _v_offsets("cuda")[slot % PAGE] + PAGE * D
    u[page[:, None, None], torch.arange(HKV, device="cuda")[None, :, None], off[:, None, :]] = vc
    scales = u[:, :, CODES:].view(torch.float32).view(s["pages"], HKV, 2, PAGE)
    scales[page, :, 0, slot % PAGE] = ks
    scales[page, :, 1, slot % PAGE] = vs
    return _appended(s, q)


# ------------------------------------------------------------------ exact

def _e4m3_values():
    """The 256 E4M3 codes by their definition: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    x = np.where(e == 0, f / 8.0 * 2.0 ** -6, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    x[(c & 0x7F) == 0x7F] = np.nan
    return torch.from_numpy(np.where(c & 128, -x, x)).cuda()


def _exact_kv(s, b, lo, hi, table):
    """K and V [8, n, 64] in 64 bits of tokens lo .. hi - 1 of sequence b, page by page."""
    pages = s["bt"][b, lo // PAGE:-(-hi // PAGE)].long()
    at = slice(lo % PAGE, lo % PAGE + hi - lo)
    if s["kv"] == "bf16":
        x = s["slab"].view(-1, 2, HKV, PAGE, D)[pages].double()
        k, v = x[:, 0], x[:, 1]
    else:
        u = s["slab"].view(-1, HKV, UNIT)[pages]
        sc = u[..., CODES:].contiguous().view(torch.float32).view(-1, HKV, 2, PAGE).double()
        codes = table[u[..., :CODES].long()]
        k = codes[..., :PAGE * D].view(-1, HKV, PAGE, D) * sc[:, :, 0, :, None]
        line = codes[..., PAGE * D:].view(-1, HKV, 8, 8, 8, 2)                # pair, stored chunk, dim, parity
        v = torch.empty_like(k)
        for p in range(8):
            for ch in range(8):
                v[:, :, 2 * p:2 * p + 2, 8 * ch:8 * ch + 8] = line[:, :, p, ch ^ (2 * p % 8)].transpose(-1, -2)
        v = v * sc[:, :, 1, :, None]
    return (x.transpose(0, 1).reshape(HKV, -1, D)[:, at] for x in (k, v))


def _exact_row(q, k, v):
    x = (q.double().view(HKV, GROUP, D) @ k.transpose(1, 2)) / 8.0
    p = torch.softmax(x, -1)
    return (p @ v).reshape(HQ, D), p


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    table = _e4m3_values()
    lens, op = s["lens"].tolist(), case["op"]
    if op in ("window", "shared", "scored"):
        out = torch.empty((s["B"], HQ, D), dtype=torch.float64, device="cuda")
        acc = s["acc"].double() if op == "scored" else None
        starts = s["starts"].tolist() if op == "shared" else []
        prefix = s["prefix"].tolist() if op == "shared" else []
        g, pk = -1, None
        for b, L in enumerate(lens):
            if op == "window":
                cut = max(0, L - case["window"])
                parts = [_exact_kv(s, b, 0, min(cut, case["sinks"]), table)] if min(cut, case["sinks"]) else []
                parts.append(_exact_kv(s, b, cut, L, table))
            elif op == "shared":
                while b >= starts[g + 1]:
                    g += 1
                    pk = tuple(_exact_kv(s, starts[g], 0, prefix[g] * PAGE, table)) if prefix[g] else None
                parts = [pk] if pk else []
                parts.append(_exact_kv(s, b, prefix[g] * PAGE, L, table))
            else:
                parts = [_exact_kv(s, b, 0, L, table)]
            k, v = (torch.cat(x, 1) for x in zip(*parts))
            out[b], p = _exact_row(s["q"][b], k, v)
            if op == "scored":
                acc[b, :, :L] += p.sum(1)
        return out if op != "scored" else {"out": out, "acc": acc}
    if op == "evict":
        return None
    # the rotation as a product of complex numbers; what is held in 8 bits has no 64-bit value
    f = torch.exp(torch.arange(D // 2, device="cuda", dtype=torch.float64) * (-2.0 / D * math.log(THETA)))
    w = torch.polar(torch.ones_like(f)[None], s["pos"].double()[:, None] * f)[:, None]
    x = s["q"].double()
    z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * w
    q = torch.cat([z.real, z.imag], -1)
    if s["kv"] == "fp8":
        return {"q": q, "codes": None, "scales": None}
    x = s["k_new"].double()
    z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * w
    pages = s["slab"].double().view(-1, 2, HKV, PAGE, D)
    for b, L in enumerate(lens):
        at = (int(s["bt"][b, (L - 1) // PAGE]), (L - 1) % PAGE)
        pages[at[0], 0, :, at[1]] = torch.cat([z[b].real, z[b].imag], -1)
        pages[at[0], 1, :, at[1]] = s["v_new"][b].double()
    return {"q": q, "pages": pages.view(-1, BF16_PAGE)}
