"""Operators for steps that bring several new tokens to a sequence, as cases to be measured.

Three operators over the paged KV cache (32 query heads, 8 KV heads of 64 dims, 16-token pages,
BF16 pages or FP8 E4M3 pages with one scale per row), used one after another in a step whose
sequences bring chunks of tokens (prompts, continued prompts) and single tokens side by side:

``tables``     block tables extended, positions and slot maps made, on the GPU, from the lengths
``append``     norms of the query and key heads, rotation (one position or three axes a token)
               and the write of the rows to their slots
``attention``  causal attention of the new tokens over their sequences' pages, optionally over
               a window and the first tokens

Where ``own`` is false ``run`` computes an operator with elementary torch operations; where it is
true it calls the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

HQ, HKV, GROUP, D, PAGE = 32, 8, 4, 64, 16
SCALE = 1.0 / math.sqrt(D)
THETA = 500000.0
EPS = 1e-5
BF16_PAGE = 2 * HKV * PAGE * D          # elements
UNIT = 2 * PAGE * (D + 4)               # bytes of one KV head of an FP8 page: codes, then row scales
CODES = 2 * PAGE * D
TOKEN_BYTES = {"bf16": 2 * HKV * D * 2, "fp8": 2 * HKV * (D + 4)}
MAX_POS = 65536                         # rows of the rotary table
AXES = (8, 12, 12)                      # rotation pairs of time, height and width


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one session takes its next token: latency of a single small call
        dict(name="tables_b1", op="tables", layers=16, batch=1, chunks=0, chunk=1, cached=700, idle=0, pad=0, ragged=1),
        # a serving step: most requests decode, some bring prompts; the arrays are those of a captured graph
        dict(name="tables_b64", op="tables", layers=16, batch=64, chunks=6, chunk=900, cached=2048, idle=3, pad=333,
             ragged=2),
        # many prompts admitted at once
        dict(name="tables_b512", op="tables", layers=16, batch=512, chunks=400, chunk=500, cached=1024, idle=20, pad=0,
             ragged=3),
        # one session's token through normed heads
        dict(name="append_t1", op="append", kv="bf16", tokens=1, pad=0, norm=True, axes=1, joint=False, ragged=4),
        # a picture and its caption: three axes, keys and values side by side as one projection leaves them
        dict(name="append_t1111_axes", op="append", kv="bf16", tokens=1111, pad=41, norm=True, axes=3, joint=True,
             ragged=5),
        # a large step of prompts into FP8 pages
        dict(name="append_t16384_fp8", op="append", kv="fp8", tokens=16384, pad=0, norm=True, axes=1, joint=True,
             ragged=6),
        # a user's next turn in one chat: latency
        dict(name="attention_b1_t33", op="attention", kv="bf16", batch=1, chunks=1, chunk=33, cached=500, idle=0,
             window=0, sinks=0, ragged=7),
        # a serving step: decoding requests with prompts among them
        dict(name="attention_b64_mixed", op="attention", kv="bf16", batch=64, chunks=8, chunk=700, cached=8192, idle=2,
             window=0, sinks=0, ragged=8),
        # fresh prompts of the engine's whole context
        dict(name="attention_b16_fresh", op="attention", kv="bf16", batch=16, chunks=16, chunk=2048, cached=0, idle=0,
             window=0, sinks=0, ragged=9),
        # single tokens only, FP8 pages: the operator as a decode step
        dict(name="attention_b200_t1_fp8", op="attention", kv="fp8", batch=200, chunks=0, chunk=1, cached=4096, idle=0,
             window=0, sinks=0, ragged=10),
        # a piece of a long document, FP8 pages
        dict(name="attention_t2048_l65000_fp8", op="attention", kv="fp8", batch=1, chunks=1, chunk=2048, cached=63000,
             idle=0, window=0, sinks=0, ragged=11),
        # long prompts of a model with a window
        dict(name="attention_b4_window", op="attention", kv="bf16", batch=4, chunks=4, chunk=4000, cached=9000, idle=0,
             window=1000, sinks=5, ragged=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_weight(c) for c in listed())
    while True:
        c = dict(op=rng.choice(["tables", "append", "attention", "attention"]), ragged=rng.randrange(100, 1 << 30))
        if c["op"] == "append":
            c.update(kv=rng.choice(["bf16", "fp8"]), tokens=_log(rng, 1, 16384), norm=rng.random() < 0.7,
                     axes=rng.choice([1, 1, 3]), joint=rng.random() < 0.5)
            c["pad"] = rng.choice([0, rng.randrange(0, c["tokens"])])
            return c
        c.update(batch=_log(rng, 1, 512 if c["op"] == "tables" else 256), cached=rng.choice([0, _log(rng, 1, 65000)]),
                 chunk=_log(rng, 1, 4096))
        c["chunks"] = rng.randrange(0, c["batch"] + 1)
        c["idle"] = rng.choice([0, rng.randrange(0, c["batch"] // 4 + 1)])
        if c["op"] == "tables":
            c.update(layers=rng.choice([1, 16, rng.randrange(1, 33)]), pad=rng.choice([0, rng.randrange(0, 1000)]))
        else:
            c["kv"] = rng.choice(["bf16", "fp8"])
            c["window"] = rng.choice([0, 0, _log(rng, 1, 4096)])
            c["sinks"] = rng.choice([0, rng.randrange(0, 65)]) if c["window"] else 0
        cached, new = _sizes(c)
        held = int((cached + new).sum()) // PAGE * c.get("layers", 1)          # pages: they bound a state's memory
        if new.sum() and _weight(c) <= most and int(new.sum()) <= 1 << 17 and held <= (1 << 18 if "layers" in c else 1 << 16):
            return c


def _sizes(case):
    """Cached lengths and new tokens of the sequences, from the case's own seed (the same for
    every input): the first `chunks` rows before a shuffle bring chunks, the last `idle` nothing."""
    r = np.random.RandomState(case["ragged"])
    B = case["batch"]
    cached = np.zeros(B, dtype=np.int64)
    if case["cached"]:
        cached = np.clip(np.rint(r.lognormal(math.log(0.4 * case["cached"]), 0.6, B)), 0, case["cached"]).astype(np.int64)
        cached[0] = case["cached"]
    new = np.ones(B, dtype=np.int64)
    n = case["chunks"]
    new[:n] = np.maximum(1, case["chunk"] * np.exp(-1.5 * r.rand(n)))
    if n:
        new[0] = case["chunk"]
    if case["idle"]:
        new[B - case["idle"]:] = 0
    at = r.permutation(B)
    return cached[at], new[at]


def _visible(case, cached, new):
    """(query, token) pairs and tokens visible to some query, over all sequences."""
    W, S = case["window"], case["sinks"]
    pairs = seen = 0
    for c, n in zip(cached.tolist(), new.tolist()):
        if not n:
            continue
        L = c + n
        if not W:
            pairs += n * c + n * (n + 1) // 2
            seen += L
            continue
        p = np.arange(c, L, dtype=np.int64)
        pairs += int((np.minimum(p + 1, W) + np.minimum(S, np.maximum(p + 1 - W, 0))).sum())
        lo = max(0, c + 1 - W)
        seen += L - lo + min(S, lo)
    return pairs, seen


def _positions(case):
    """Positions [axes][tokens] of the valid tokens from 0 on: text, then (three axes) a picture of
    rows and columns at one time."""
    n = case["tokens"] - case["pad"]
    t = np.arange(n)
    if case["axes"] == 1:
        return t[None]
    text = n // 5
    side = max(1, int(math.sqrt(max(1, n - text))))
    i = np.maximum(t - text, 0)
    picture = t >= text
    return np.stack([np.where(picture, text, t), np.where(picture, text + i // side, t),
                     np.where(picture, text + i % side, t)])


def work(case):
    if case["op"] == "append":
        n = case["tokens"] - case["pad"]
        pairs = (D // 2,) if case["axes"] == 1 else AXES
        table = sum(len(np.unique(p)) * k * 16 for p, k in zip(_positions(case), pairs))
        per = HQ * D * 2 * 2 + 2 * HKV * D * 2 + TOKEN_BYTES[case["kv"]] + 8 + 4 * case["axes"]
        return {"bytes": n * per + table + 8 * case["pad"] + (2 * D * 2 if case["norm"] else 0),
                "flops": n * (HQ + HKV) * D * (3 + (4 if case["norm"] else 0))}
    cached, new = _sizes(case)
    T = int(new.sum())
    if case["op"] == "tables":
        fresh = int((-(-(cached + new) // PAGE) + (-cached // PAGE)).sum()) * case["layers"]
        part = int(((cached % PAGE > 0) & (new > 0)).sum()) * case["layers"]
        n = T + case["pad"]
        return {"bytes": 8 * case["batch"] + 4 * part + 8 * fresh + n * (4 + 8 * case["layers"]) + 8 * case["batch"] + 12,
                "flops": 0}
    pairs, seen = _visible(case, cached, new)
    return {"bytes": seen * TOKEN_BYTES[case["kv"]] + T * HQ * D * 2 * 2, "flops": 4 * D * HQ * pairs}


def _weight(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 100)


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


def _fill_pages(kv, pages, gen):
    """A slab of pages of N(0, 1) rows, one key row in a hundred eight times as large."""
    slab = torch.empty(pages * BF16_PAGE, dtype=torch.bfloat16, device="cuda") if kv == "bf16" else \
        torch.empty(pages * HKV * UNIT, dtype=torch.uint8, device="cuda")
    off = _v_offsets("cuda").reshape(-1)
    step = 8192
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = torch.randn((n, HKV, 2, PAGE, D), generator=gen, device="cuda")
        x[:, :, 0] *= torch.where(torch.rand((n, HKV, PAGE, 1), generator=gen, device="cuda") < 0.01, 8.0, 1.0)
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

def _int(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    s = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    {"tables": _prepare_tables, "append": _prepare_append, "attention": _prepare_attention}[case["op"]](s, case, gen, r)
    if own:
        _own_handles(s)
    return s


def _prepare_tables(s, case, gen, r):
    cached, new = _sizes(case)
    layers, B = case["layers"], case["batch"]
    had, need = -(-cached // PAGE), -(-(cached + new) // PAGE)
    blocks = int(need.max()) + 3
    held, fresh = layers * int(had.sum()), layers * int((need - had).sum())
    spare = 5 + fresh // 4
    ids = r.permutation(held + fresh + spare + 7).astype(np.int32)
    bt = np.full((layers, B, blocks), -1, dtype=np.int32)
    bt[np.broadcast_to(np.arange(blocks)[None, None, :] < had[None, :, None], bt.shape)] = ids[:held]
    T = int(new.sum()) + case["pad"]
    # the list of pages to take from, of which earlier steps have used up a few
    s.update(layers=layers, B=B, blocks=blocks, T=T, total=int(new.sum()), num_pages=len(ids), bt=_int(bt), lens=_int(cached),
             new=_int(new), pages=_int(ids[held:]), used=_int([3]),
             starts=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
             lens_out=torch.zeros(B, dtype=torch.int32, device="cuda"),
             used_out=torch.zeros(1, dtype=torch.int32, device="cuda"),
             pos=torch.zeros(T, dtype=torch.int32, device="cuda"),
             slots=torch.zeros((layers, T), dtype=torch.int64, device="cuda"))


def _prepare_append(s, case, gen, r):
    T, n = case["tokens"], case["tokens"] - case["pad"]
    kv = case["kv"]
    first = int(r.randint(0, PAGE))                   # the chunk begins inside a page
    pages = (first + n + PAGE - 1) // PAGE + 2
    at = first + np.arange(n)
    slots = np.full(T, -1, dtype=np.int64)
    slots[:n] = r.permutation(pages)[at // PAGE].astype(np.int64) * PAGE + at % PAGE
    pos = np.zeros((case["axes"], T), dtype=np.int64)
    p = _positions(case)
    pos[:, :n] = p + r.randint(0, MAX_POS - (int(p.max()) if n else 0))
    s.update(kv=kv, T=T, pages=pages, slab=_fill_pages(kv, pages, gen), slots=_int(slots, torch.int64), pos=_int(pos))

    def rows(shape):
        # projections: tokens and heads of different sizes
        x = torch.randn(shape, generator=gen, device="cuda")
        x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen, device="cuda"))
        return x.to(torch.bfloat16)

    s["q"] = rows((T, HQ, D))
    if case["joint"]:
        both = rows((T, 2, HKV, D))
        s["k"], s["v"] = both[:, 0], both[:, 1]
    else:
        s["k"], s["v"] = rows((T, HKV, D)), rows((T, HKV, D))
    s["q_out"] = torch.zeros((T, HQ, D), dtype=torch.bfloat16, device="cuda")
    s["qw"] = s["kw"] = None
    if case["norm"]:
        s["qw"], s["kw"] = ((1.0 + 0.3 * torch.randn(D, generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2))


def _prepare_attention(s, case, gen, r):
    cached, new = _sizes(case)
    B, lens = case["batch"], cached + new
    need = -(-lens // PAGE)
    blocks = max(1, int(need.max()))
    pages = max(1, int(need.sum()))
    bt = np.full((B, blocks), -1, dtype=np.int32)
    bt[np.arange(blocks)[None, :] < need[:, None]] = r.permutation(int(need.sum())).astype(np.int32)
    T = int(new.sum())
    starts = np.concatenate([[0], np.cumsum(new)])
    s.update(kv=case["kv"], B=B, T=T, blocks=blocks, pages=pages, slab=_fill_pages(case["kv"], pages, gen), bt=_int(bt),
             lens=_int(lens), starts=_int(starts), rows=list(zip(starts.tolist(), new.tolist(), lens.tolist())),
             q=torch.randn((T, HQ, D), generator=gen, device="cuda").to(torch.bfloat16))
    s["out"] = torch.zeros_like(s["q"])


def _own_handles(s):
    """The pool object, the workspace and the rotary table that a user's program keeps."""
    from paged_kv_decode_12_gb300 import pkv

    op = s["case"]["op"]
    ws = 0
    if op == "tables":
        # (the call only asks the pool how many pages it has)
        s["slab"] = torch.empty(s["num_pages"] * HKV * UNIT, dtype=torch.uint8, device="cuda")
        s["pool"] = pkv.pkv_pool_create_fp8(s["slab"], s["slab"].numel())
        ws = pkv.pkv_chunk_tables_workspace_bytes(s["B"])
    else:
        make = pkv.pkv_pool_create if s["kv"] == "bf16" else pkv.pkv_pool_create_fp8
        s["pool"] = make(s["slab"], s["slab"].numel() * s["slab"].element_size())
    if op == "append":
        s["rope"] = pkv.rope_table(MAX_POS, "cuda", THETA)
    elif op == "attention":
        ws = pkv.pkv_chunk_attention_workspace_bytes(s["B"], s["T"])
    s["ws"], s["ws_bytes"] = torch.zeros(max(ws, 16), dtype=torch.uint8, device="cuda"), ws


# ------------------------------------------------------------------ run

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from paged_kv_decode_12_gb300 import pkv

    case = s["case"]
    if case["op"] == "tables":
        pkv.pkv_chunk_tables(s["pool"], s["lens"], s["new"], s["B"], s["bt"], s["blocks"], s["layers"], s["pages"],
                             s["pages"].numel(), s["used"], s["used_out"], s["T"], s["starts"], s["lens_out"], s["pos"],
                             s["slots"], s["ws"], s["ws_bytes"], s["err"])
        return _tables(s)
    if case["op"] == "append":
        pkv.pkv_chunk_append(s["pool"], s["k"], s["k"].stride(0), s["v"], s["v"].stride(0), s["q"], s["q"].stride(0),
                             s["q_out"], s["qw"], s["kw"], EPS, s["slots"], s["pos"], s["T"],
                             AXES if case["axes"] == 3 else None, s["T"], s["rope"], MAX_POS, s["err"])
        return _appended(s)
    pkv.pkv_chunk_attention(s["pool"], s["q"], s["bt"], s["blocks"], s["lens"], s["starts"], s["B"], s["T"], SCALE,
                            case["window"], case["sinks"], s["ws"], s["ws_bytes"], s["out"], s["err"])
    return s["out"]


def _run_plain(s):
    return {"tables": _plain_tables, "append": _plain_append, "attention": _plain_attention}[s["case"]["op"]](s)


def _tables(s):
    return {"bt": s["bt"], "starts": s["starts"], "lens": s["lens_out"], "used": s["used_out"], "pos": s["pos"],
            "slots": s["slots"]}


def _plain_tables(s):
    lens, new, layers, B, T = s["lens"].long(), s["new"].long(), s["layers"], s["B"], s["T"]
    had, need = (lens + PAGE - 1) // PAGE, (lens + new + PAGE - 1) // PAGE
    fresh = need - had
    before, total = torch.cumsum(fresh, 0) - fresh, fresh.sum()
    # new pages: layer by layer, sequence by sequence
    j = torch.arange(s["blocks"], device="cuda")
    mine = (j >= had[:, None]) & (j < need[:, None])
    place = s["used"].long() + before[:, None] + j - had[:, None] + total * torch.arange(layers, device="cuda")[:, None, None]
    place = torch.where(mine, place, 0)
    s["bt"].copy_(torch.where(mine, s["pages"][place], s["bt"]))
    s["starts"][1:] = torch.cumsum(new, 0)
    s["lens_out"].copy_(lens + new)
    s["used_out"].copy_(s["used"] + total * layers)
    # every new token's position and slot; none behind the last
    row = torch.repeat_interleave(torch.arange(B, device="cuda"), new, output_size=s["total"])
    n = s["total"]
    p = lens[row] + torch.arange(n, device="cuda") - s["starts"][row]
    s["pos"][:n] = p
    s["pos"][n:] = 0
    s["slots"][:, :n] = s["bt"][:, row, p // PAGE].long() * PAGE + p % PAGE
    s["slots"][:, n:] = -1
    return _tables(s)


def _appended(s):
    out = {"q": s["q_out"]}
    if s["kv"] == "bf16":
        out["pages"] = s["slab"]
    else:
        u = s["slab"].view(s["pages"], HKV, UNIT)
        out.update(codes=u[:, :, :CODES].view(torch.float8_e4m3fn), scales=u[:, :, CODES:].view(torch.float32))
    return out


def _plain_append(s):
    # (in 64 bits: angles of far positions, and sums next to a rounding border)
    i = torch.arange(D // 2, device="cuda", dtype=torch.float64)
    axis = torch.zeros(D // 2, dtype=torch.long, device="cuda") if s["case"]["axes"] == 1 else \
        torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(AXES, device="cuda"), output_size=D // 2)
    angle = s["pos"].double().t()[:, axis] * THETA ** (-2.0 * i / D)
    c, z = torch.cos(angle)[:, None], torch.sin(angle)[:, None]

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()
        x1, x2 = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([x1 * c - x2 * z, x2 * c + x1 * z], -1).to(torch.bfloat16)

    q, k = turned(s["q"], s["qw"]), turned(s["k"], s["kw"])
    there = s["slots"] >= 0
    s["q_out"].copy_(torch.where(there[:, None, None], q, s["q_out"]))
    at = torch.nonzero(there)[:, 0]
    page, slot = s["slots"][at] // PAGE, s["slots"][at] % PAGE
    if s["kv"] == "bf16":
        x = s["slab"].view(s["pages"], 2, HKV, PAGE, D)
        x[page, 0, :, slot] = k[at]
        x[page, 1, :, slot] = s["v"][at]
        return _appended(s)
    u = s["slab"].view(s["pages"], HKV, UNIT)
    kc, ks = _quantize(k[at].float())
    vc, vs = _quantize(s["v"][at].float())
    u[:, :, :PAGE * D].view(s["pages"], HKV, PAGE, D)[page, :, slot] = kc
    off = _v_offsets("cuda")[slot] + PAGE * D
    u[page[:, None, None], torch.arange(HKV, device="cuda")[None, :, None], off[:, None, :]] = vc
    scales = u[:, :, CODES:].view(torch.float32).view(s["pages"], HKV, 2, PAGE)
    scales[page, :, 0, slot] = ks
    scales[page, :, 1, slot] = vs
    return _appended(s)


def _gather(s, b, tokens):
    """K and V [8, n, 64] in FP32 of tokens of sequence b."""
    page, slot = s["bt"][b, tokens // PAGE].long(), tokens % PAGE
    if s["kv"] == "bf16":
        x = s["slab"].view(s["pages"], 2, HKV, PAGE, D)[page, :, :, slot].float()
        return x[:, 0].transpose(0, 1), x[:, 1].transpose(0, 1)
    u = s["slab"].view(s["pages"], HKV, UNIT)
    scales = u[:, :, CODES:].view(torch.float32).view(s["pages"], HKV, 2, PAGE)[page, :, :, slot]
    kc = u[:, :, :PAGE * D].view(s["pages"], HKV, PAGE, D)[page, :, slot]
    head = torch.arange(HKV, device="cuda")[:, None]
    off = _v_offsets("cuda")[slot][:, None, :] + PAGE * D
    vc = u[page[:, None, None], head, off]
    k = kc.view(torch.float8_e4m3fn).float() * scales[:, :, 0, None]
    v = vc.view(torch.float8_e4m3fn).float() * scales[:, :, 1, None]
    return k.transpose(0, 1), v.transpose(0, 1)


def _plain_attention(s):
    W, S = s["case"]["window"], s["case"]["sinks"]
    for b, (t0, n, L) in enumerate(s["rows"]):
        if not n:
            continue
        lo = max(0, L - n + 1 - W) if W else 0
        t = torch.arange(lo, L, device="cuda")
        if lo and S:
            t = torch.cat([torch.arange(min(S, lo), device="cuda"), t])
        k, v = _gather(s, b, t)
        step = max(1, (1 << 28) // (HQ * t.numel()))           # (scores of a gigabyte at a time)
        for i in range(0, n, step):
            m = min(step, n - i)
            q = s["q"][t0 + i:t0 + i + m].float().view(m, HKV, GROUP, D).permute(1, 2, 0, 3)   # [8, 4, m, 64]
            x = (q.reshape(HKV, GROUP * m, D) @ k.transpose(1, 2)).view(HKV, GROUP, m, -1) * SCALE
            p = torch.arange(L - n + i, L - n + i + m, device="cuda")[:, None]
            seen = t <= p
            if W:
                seen &= (t > p - W) | (t < S)
            x = x.masked_fill(~seen, -math.inf)
            e = torch.exp(x - x.amax(-1, keepdim=True))
            e = e / e.sum(-1, keepdim=True)
            o = (e.view(HKV, GROUP * m, -1) @ v).view(HKV, GROUP, m, D)
            s["out"][t0 + i:t0 + i + m] = o.permute(2, 0, 1, 3).reshape(m, HQ, D).to(torch.bfloat16)
    return s["out"]


# ------------------------------------------------------------------ exact

def _e4m3_values():
    """The 256 E4M3 codes by their definition: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    x = np.where(e == 0, f / 8.0 * 2.0 ** -6, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    x[(c & 0x7F) == 0x7F] = np.nan
    return torch.from_numpy(np.where(c & 128, -x, x)).cuda()


def _exact_cache(s, b, L, table):
    """K and V [8, L, 64] in 64 bits of sequence b, page by page."""
    pages = s["bt"][b, :-(-L // PAGE)].long()
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
    return (x.transpose(0, 1).reshape(HKV, -1, D)[:, :L] for x in (k, v))


def exact(case, seed):
    global own
    if case["op"] == "tables":
        return None
    was, own = own, False
    s = prepare(case, seed)
    own = was
    return (_exact_attention if case["op"] == "attention" else _exact_append)(s, case)


def _exact_attention(s, case):
    if work(case)["flops"] > 6e12:
        return None
    table = _e4m3_values()
    out = torch.zeros((s["T"], HQ, D), dtype=torch.float64, device="cuda")
    at = 0
    for b in range(s["B"]):
        L = int(s["lens"][b])
        n = int(s["starts"][b + 1]) - int(s["starts"][b])
        if n == 0:
            continue
        k, v = _exact_cache(s, b, L, table)
        for g in range(HKV):
            step = max(1, (1 << 25) // L)
            for i in range(0, n, step):
                m = min(step, n - i)
                last = L - n + i + torch.arange(m, device="cuda")
                dist = last[:, None] - torch.arange(L, device="cuda")[None, :]
                hidden = dist < 0
                if case["window"]:
                    hidden |= (dist >= case["window"]) & (torch.arange(L, device="cuda")[None, :] >= case["sinks"])
                for h in range(g * GROUP, (g + 1) * GROUP):
                    x = s["q"][at + i:at + i + m, h].double() @ k[g].t() / 8.0
                    x[hidden] = -math.inf
                    out[at + i:at + i + m, h] = torch.softmax(x, -1) @ v[g]
        at += n
    return out


def _exact_append(s, case):
    # the rotation as a product of complex numbers; what is held in 8 bits has no 64-bit value
    n = case["tokens"] - case["pad"]
    f = torch.exp(torch.arange(D // 2, device="cuda", dtype=torch.float64) * (-2.0 / D * math.log(THETA)))
    if case["axes"] == 1:
        angle = s["pos"][0, :n, None].double() * f
    else:
        parts, first = [], 0
        for a, pairs in enumerate(AXES):
            parts.append(s["pos"][a, :n, None].double() * f[first:first + pairs])
            first += pairs
        angle = torch.cat(parts, 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rows(x, w):
        x = x[:n].double()
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS) * w.double()
        z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * turn
        return torch.cat([z.real, z.imag], -1)

    q = s["q_out"].double()
    q[:n] = rows(s["q"], s["qw"])
    if s["kv"] == "fp8":
        return {"q": q, "codes": None, "scales": None}
    pages = s["slab"].double().view(-1, 2, HKV, PAGE, D)
    at = s["slots"][:n]
    pages[at // PAGE, 0, :, at % PAGE] = rows(s["k"], s["kw"])
    pages[at // PAGE, 1, :, at % PAGE] = s["v"][:n].double()
    return {"q": q, "pages": pages.view(-1)}
