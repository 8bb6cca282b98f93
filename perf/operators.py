"""Serving operators around the verify step: an 8-bit KV cache (written, read
back, attended to) and log probabilities from the LM head.

``listed()`` and ``draw()`` give cases, ``prepare()`` makes what a serving
program holds before the call, ``run()`` makes one call: in elementary torch
operations, or, with ``own`` set, through the library's entry points.

The cache holds codes c and, for every block of positions and every head, the
largest magnitude a of the block; a code stands for c * a / Q, Q = 127 (int8) or
448 (e4m3). Inside each group of 16 positions the codes lie in the order in
which the attention's tensor-core operands read them:

    key   (p, d): [p / 16][d / 64][p % 16][d % 64]
    value (p, d): [p / 16][d / 4][p % 16 / 4][d % 4][p % 4]
"""
import math

import torch

own = False  # True: run() calls the library

DEV = "cuda"
Q_OF = {"int8": 127.0, "e4m3": 448.0}
CODE_OF = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}

VOCAB, HIDDEN, HEADS, DIM = 129280, 1280, 10, 128  # the decoder's own sizes


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence's verify step: 4 new rows into a short cache, latency only
        {"name": "write-b1", "op": "write", "format": "int8", "B": 1, "rows": 4, "n_kv": HEADS, "dim": DIM, "block": 64,
         "pos": 777, "ragged": 0.0, "back": "fp32"},
        # the batched verify step: 32 sequences x 4 rows, ragged lengths around 2,048
        {"name": "write-b32-e4m3", "op": "write", "format": "e4m3", "B": 32, "rows": 4, "n_kv": HEADS, "dim": DIM, "block": 32,
         "pos": 2048, "ragged": 0.4, "back": "fp32"},
        # pages of prompt written at once (padded batch), then handed on in bf16
        {"name": "write-prompt", "op": "write", "format": "int8", "B": 4, "rows": 8191, "n_kv": HEADS, "dim": DIM, "block": 64,
         "pos": 0, "ragged": 0.5, "back": "bf16"},
        # one short sequence read back for inspection
        {"name": "read-b1", "op": "read", "format": "int8", "B": 1, "rows": 301, "n_kv": HEADS, "dim": DIM, "block": 64,
         "pos": 5, "ragged": 0.0, "back": "fp32"},
        # a batch moved back to a bf16 cache
        {"name": "read-b8-e4m3", "op": "read", "format": "e4m3", "B": 8, "rows": 8190, "n_kv": HEADS, "dim": DIM, "block": 32,
         "pos": 0, "ragged": 0.3, "back": "bf16"},
        # one sequence's verify step early in a page
        {"name": "attn-b1", "op": "attn", "format": "int8", "B": 1, "rows": 4, "heads": HEADS, "n_kv": HEADS, "dim": DIM,
         "block": 64, "len": 777, "ragged": 0.0, "window": 0},
        # the batched verify step at 2,048 cached positions
        {"name": "attn-b32-l2048", "op": "attn", "format": "int8", "B": 32, "rows": 4, "heads": HEADS, "n_kv": HEADS,
         "dim": DIM, "block": 64, "len": 2048, "ragged": 0.4, "window": 0},
        # shared key/value heads, long ragged caches with their oldest positions dropped
        {"name": "attn-b32-shared-e4m3", "op": "attn", "format": "e4m3", "B": 32, "rows": 4, "heads": 32, "n_kv": 8,
         "dim": DIM, "block": 32, "len": 12289, "ragged": 0.6, "window": 8192},
        # the longest caches the decoder allows, the most new rows
        {"name": "attn-b16-l32760", "op": "attn", "format": "int8", "B": 16, "rows": 8, "heads": HEADS, "n_kv": HEADS,
         "dim": DIM, "block": 128, "len": 32760, "ragged": 0.0, "window": 0},
        # one sequence's committed tokens with five alternatives
        {"name": "logprob-r4", "op": "logprob", "R": 4, "H": HIDDEN, "V": VOCAB, "top": 5},
        # the batched verify step's 128 rows with twenty alternatives
        {"name": "logprob-r128", "op": "logprob", "R": 128, "H": HIDDEN, "V": VOCAB, "top": 20},
        # scoring whole pages: 4,096 rows
        {"name": "logprob-r4096", "op": "logprob", "R": 4096, "H": HIDDEN, "V": VOCAB, "top": 5},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "logprob", "logprob"])
    if op == "logprob":
        R = _log(rng, 1, 4096)
        H = 64 * _log(rng, 4, 32)
        V = _log(rng, 1000, 160000)
        if R * H * V > 4096 * HIDDEN * VOCAB:
            R = max(1, 4096 * HIDDEN * VOCAB // (H * V))
        return {"op": op, "R": R, "H": H, "V": V, "top": rng.choice([0, 1, 5, rng.randint(2, 20)])}
    fmt, dim, block = rng.choice(["int8", "e4m3"]), rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    n_kv = rng.choice([1, 2, 4, 8, 10])
    B = _log(rng, 1, 64)
    if op == "attn":
        L = _log(rng, 1, 32000)
        B = max(1, min(B, 16 * 32768 * HEADS * DIM // (2 * L * n_kv * dim)))
        return {"op": op, "format": fmt, "B": B, "rows": rng.randint(1, 8), "heads": n_kv * rng.choice([1, 1, 2, 4, 8]),
                "n_kv": n_kv, "dim": dim, "block": block, "len": L, "ragged": rng.choice([0.0, 0.5, 0.9]),
                "window": rng.choice([0, 0, 0, _log(rng, 1, 8192)])}
    rows = _log(rng, 1, 8192) if op == "read" or rng.random() < 0.5 else rng.randint(1, 8)
    B = max(1, min(B, 4 * 8192 * HEADS * DIM // (2 * rows * n_kv * dim)))
    return {"op": op, "format": fmt, "B": B, "rows": rows, "n_kv": n_kv, "dim": dim, "block": block,
            "pos": rng.choice([0, _log(rng, 1, 4096)]), "ragged": rng.choice([0.0, 0.5]), "back": rng.choice(["bf16", "fp32"])}


# ------------------------------------------------------------------ sizes that follow from a case
def _up(n, m):
    return (n + m - 1) // m * m


def _spread(top, ragged, B, step):
    """top for the first sequence, down to (1 - ragged) * top for others."""
    span = int(top * ragged) + 1
    return [top - (b * step) % span for b in range(B)]


def _attn_lens(c):
    lens = _spread(c["len"], c["ragged"], c["B"], 977)
    first = [max(0, n + 1 - c["window"]) for n in lens] if c["window"] else [0] * c["B"]
    return lens, first, _up(c["len"] + c["rows"], c["block"])


def _row_counts(c):
    pos = _spread(c["pos"], c["ragged"], c["B"], 977)
    n = [max(1, x) for x in _spread(c["rows"], c["ragged"], c["B"], 613)]
    return pos, n, _up(c["pos"] + c["rows"], c["block"])


# ------------------------------------------------------------------ cache layout
def _pack_k(x):
    B, h, L, D = x.shape
    return x.view(B, h, L // 16, 16, D // 64, 64).transpose(3, 4).contiguous().view(B, h, L, D)


def _unpack_k(x):
    B, h, L, D = x.shape
    return x.view(B, h, L // 16, D // 64, 16, 64).transpose(3, 4).reshape(B, h, L, D)


def _pack_v(x):
    B, h, L, D = x.shape
    return x.view(B, h, L // 16, 4, 4, D // 4, 4).permute(0, 1, 2, 5, 3, 6, 4).contiguous().view(B, h, L, D)


def _unpack_v(x):
    B, h, L, D = x.shape
    return x.view(B, h, L // 16, D // 4, 4, 4, 4).permute(0, 1, 2, 4, 6, 3, 5).reshape(B, h, L, D)


def _bytes(x):
    return x.view(torch.uint8)  # moving codes needs no arithmetic type


def _encode(x, fmt):
    """Values x Q / a, already formed, to codes: to the nearest, ties to even."""
    return torch.round(x).to(torch.int8) if fmt == "int8" else x.to(torch.float8_e4m3fn)


def _decode(c, a, block, fmt, dtype):
    """[B, h, L, D] codes in order, [B, h, L / block] -> values c a / Q."""
    a = a.to(dtype).repeat_interleave(block, 2)[..., None]
    q = torch.full((), Q_OF[fmt], dtype=dtype, device=c.device)
    return c.to(dtype) * a / q


def _fill(gen, B, h, L, D, block, fmt, kind):
    """A cache's codes and magnitudes for normal values whose channels differ in
    size (keys: a few channels ten times the others)."""
    codes = torch.empty(B, h, L, D, dtype=CODE_OF[fmt], device=DEV)
    amax = torch.empty(B, h, L // block, device=DEV)
    size = torch.rand(h, 1, D, generator=gen, device=DEV) * 0.7 + 0.3
    if kind == "k":
        size = size * torch.where(torch.rand(h, 1, D, generator=gen, device=DEV) < 0.03, 6.0, 1.0)
    for b in range(B):
        x = (torch.randn(h, L, D, generator=gen, device=DEV) * size).bfloat16().float().view(h, L // block, block, D)
        a = x.abs().amax((2, 3))
        code = _encode(x * Q_OF[fmt] / a[..., None, None], fmt).view(1, h, L, D)
        codes[b] = (_pack_k if kind == "k" else _pack_v)(_bytes(code)).view(CODE_OF[fmt])[0]
        amax[b] = a
    return codes, amax


# ------------------------------------------------------------------ what a program holds
def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    s = {"case": dict(c)}
    if c["op"] == "logprob":
        R, H, V = c["R"], c["H"], c["V"]
        lm = torch.empty(V, H, dtype=torch.bfloat16, device=DEV)
        for i in range(0, V, 16384):
            lm[i:i + 16384] = (randn(min(16384, V - i), H) * (1.2 / math.sqrt(H))).bfloat16()
        tok = torch.randint(0, V, (R,), generator=gen, device=DEV, dtype=torch.int32)
        # rows from undecided (all noise) to certain (one token far above the others)
        sure = torch.rand(R, 1, generator=gen, device=DEV) * 14.0
        h = randn(R, H) + sure * torch.nn.functional.normalize(lm[tok.long()].float(), dim=1)
        tok[1::3] = torch.randint(0, V, (R,), generator=gen, device=DEV, dtype=torch.int32)[1::3]  # and unlikely tokens
        s.update(lm=lm, h=h.bfloat16(), tok=tok, logprob=torch.zeros(R, device=DEV), entropy=torch.zeros(R, device=DEV),
                 ids=torch.zeros(R, c["top"], dtype=torch.int32, device=DEV), top=torch.zeros(R, c["top"], device=DEV))
        return s
    B, h, D, block, fmt = c["B"], c["n_kv"], c["dim"], c["block"], c["format"]
    if c["op"] == "attn":
        lens, first, L = _attn_lens(c)
        s["k"], s["ka"] = _fill(gen, B, h, L, D, block, fmt, "k")
        s["v"], s["va"] = _fill(gen, B, h, L, D, block, fmt, "v")
        s.update(q=(randn(B * c["rows"], c["heads"] * D) * 1.5).bfloat16(), lens=ints(lens), first=ints(first),
                 scale=1.0 / math.sqrt(D), o=torch.zeros(B * c["rows"], c["heads"] * D, dtype=torch.bfloat16, device=DEV))
        return s
    pos, n, L = _row_counts(c)
    out = torch.bfloat16 if c["back"] == "bf16" else torch.float32
    if c["op"] == "write":
        # the step before left positions 0 .. pos - 1; rows come as columns of one [rows, 3 h D] projection
        s["k"], s["ka"] = _fill(gen, B, h, L, D, block, fmt, "k")
        s["v"], s["va"] = _fill(gen, B, h, L, D, block, fmt, "v")
        big = 1.0 + torch.rand(B * c["rows"], 1, generator=gen, device=DEV)
        s["qkv"] = (randn(B * c["rows"], 3 * h * D) * big).bfloat16()
        # read back from the start of the first block that the call may recode
        back = [p // block * block for p in pos]
        rows_back = c["rows"] + block - 1
        s.update(pos=ints(pos), n=ints(n), back=ints(back), n_back=ints([p + m - q for p, m, q in zip(pos, n, back)]),
                 rows_back=rows_back)
    else:
        s["k"], s["ka"] = _fill(gen, B, h, L, D, block, fmt, "k")
        s["v"], s["va"] = _fill(gen, B, h, L, D, block, fmt, "v")
        s.update(back=ints(pos), n_back=ints(n), rows_back=c["rows"])
    s["k_out"] = torch.zeros(B * s["rows_back"], h * D, dtype=out, device=DEV)
    s["v_out"] = torch.zeros(B * s["rows_back"], h * D, dtype=out, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _own_logprob(s) if op == "logprob" else _own_attn(s) if op == "attn" else _own_cache(s)
    if op == "logprob":
        return _plain_logprob(s)
    if op == "attn":
        return _plain_attn(s)
    if op == "write":
        _plain_write(s["case"], s["qkv"], s["k"], s["ka"], s["pos"], s["n"], 1, _unpack_k, _pack_k)
        _plain_write(s["case"], s["qkv"], s["v"], s["va"], s["pos"], s["n"], 2, _unpack_v, _pack_v)
    out = {"k": _plain_read(s, s["k"], s["ka"], _unpack_k, s["k_out"]), "v": _plain_read(s, s["v"], s["va"], _unpack_v, s["v_out"])}
    return {**out, "k_amax": s["ka"], "v_amax": s["va"]} if op == "write" else out


def _handle(s):
    """The cache handle that a program keeps beside its tensors."""
    if "handle" not in s:
        import greedy_speculative_verify_b200 as vgv

        s["lib"] = vgv
        s["handle"] = vgv.make_kv8(s["k"], s["v"], s["ka"], s["va"])
    return s["lib"], s["handle"]


def _own_cache(s):
    vgv, kv = _handle(s)
    c = s["case"]
    if c["op"] == "write":
        w = c["n_kv"] * c["dim"]
        vgv.vg_kv8_append(kv, c["rows"], s["qkv"][:, w:2 * w], s["qkv"][:, 2 * w:], s["pos"], n_new=s["n"])
    vgv.vg_kv8_read(kv, s["rows_back"], s["back"], s["k_out"], s["v_out"], n_rows=s["n_back"])
    out = {"k": s["k_out"], "v": s["v_out"]}
    return {**out, "k_amax": s["ka"], "v_amax": s["va"]} if c["op"] == "write" else out


def _own_attn(s):
    vgv, kv = _handle(s)
    c = s["case"]
    if "ws" not in s:  # zero-filled once, as the call wants it
        s["ws"] = torch.zeros(max(16, vgv.vg_kv8_attn_workspace_bytes(kv, c["rows"], c["heads"])), dtype=torch.uint8, device=DEV)
    vgv.vg_kv8_attn(kv, c["rows"], c["heads"], s["q"], s["lens"], s["scale"], s["o"], s["ws"],
                    first=s["first"] if c["window"] else None)
    return s["o"]


def _own_logprob(s):
    import greedy_speculative_verify_b200 as vgv

    c = s["case"]
    if "ws" not in s:
        s["ws"] = torch.zeros(vgv.vg_token_logprobs_workspace_bytes(c["R"], c["H"], c["V"], c["top"]), dtype=torch.uint8,
                              device=DEV)
    ids, top = (s["ids"], s["top"]) if c["top"] else (None, None)
    vgv.vg_token_logprobs(s["h"], s["lm"], s["tok"], s["logprob"], s["entropy"], ids, top, s["ws"])
    return {"logprob": s["logprob"], "entropy": s["entropy"], "ids": s["ids"], "top": s["top"]}


# ------------------------------------------------------------------ plain forms
def _plain_write(c, qkv, codes, amax, pos, n, part, unpack, pack):
    """Rows i < n[b] of the part-th third of qkv to positions pos[b] + i. A block
    that already holds earlier positions keeps its magnitude or takes a larger
    one, and its earlier codes are rounded again for it; a block whose first
    position is written takes the magnitude of the new rows."""
    B, rows, h, D, block, fmt = c["B"], c["rows"], c["n_kv"], c["dim"], c["block"], c["format"]
    L = codes.shape[2]
    w = h * D
    x = qkv[:, part * w:(part + 1) * w].float().view(B, rows, h, D)
    nb = (rows + block - 2) // block + 1  # blocks that rows consecutive positions can touch
    pos, n = pos.long(), n.long()
    blk0 = pos // block
    # the window of nb blocks from blk0, as rows of new values
    at = blk0[:, None] * block + torch.arange(nb * block, device=x.device)  # [B, nb block] positions
    i = at - pos[:, None]
    new = (i >= 0) & (i < n[:, None])
    xw = x.gather(1, i.clamp(0, rows - 1)[..., None, None].expand(-1, -1, h, D))
    xw = torch.where(new[..., None, None], xw, torch.zeros_like(xw)).permute(0, 2, 1, 3)  # [B, h, nb block, D]
    a_new = xw.abs().reshape(B, h, nb, block * D).amax(3)
    bi = (blk0[:, None] + torch.arange(nb, device=x.device))
    touched = new.view(B, nb, block).any(2)
    bi_in = bi.clamp(max=L // block - 1)[:, None].expand(-1, h, -1)
    a_old = amax.gather(2, bi_in)
    holds = (torch.arange(nb, device=x.device) == 0) & (pos % block > 0)[:, None]  # only the first block can
    a_was = torch.where(holds[:, None], a_old, torch.zeros_like(a_old))
    a = torch.maximum(a_was, a_new)
    q = torch.full((), Q_OF[fmt], device=x.device)
    a_safe = torch.where(a > 0, a, torch.ones_like(a)).repeat_interleave(block, 2)[..., None]
    fresh = _bytes(_encode(xw * q / a_safe, fmt))
    at_in = at.clamp(max=L - 1)
    whole = unpack(_bytes(codes))
    old = whole.gather(2, at_in[:, None, :, None].expand(-1, h, -1, D))
    turned = old.view(codes.dtype).float() * a_was.repeat_interleave(block, 2)[..., None] / a_safe
    grown = (a > a_was)[:, :, :1] & holds[:, :1, None].transpose(1, 2)
    turn = (i < 0)[:, None, :, None] & grown.repeat_interleave(nb * block, 2)[..., None]
    put = torch.where(new[:, None, :, None], fresh, torch.where(turn, _bytes(_encode(turned, fmt)), old))
    keep = (at < L)[:, None, :, None].expand(-1, h, -1, D)
    b_i, h_i = torch.arange(B, device=x.device)[:, None, None], torch.arange(h, device=x.device)[None, :, None]
    at_all = torch.where(keep[..., 0], at[:, None, :].expand(-1, h, -1), torch.full_like(at, L)[:, None].expand(-1, h, -1))
    whole = torch.cat([whole, whole[:, :, :1]], 2)  # positions behind the cache land in a row that is dropped
    whole[b_i.expand_as(at_all), h_i.expand_as(at_all), at_all] = put
    codes.copy_(pack(whole[:, :, :L].contiguous()).view(codes.dtype))
    a_all = torch.where(touched[:, None].expand_as(a), bi[:, None].expand_as(a), torch.full_like(a, L // block).long())
    wide = torch.cat([amax, amax[:, :, :1]], 2)
    wide[b_i.expand_as(a_all), h_i.expand_as(a_all), a_all] = a
    amax.copy_(wide[:, :, :L // block])


def _plain_read(s, codes, amax, unpack, out):
    c = s["case"]
    rows, back, n = s["rows_back"], s["back"].long(), s["n_back"].long()
    B, h, L, D = codes.shape
    i = torch.arange(rows, device=codes.device)
    at = (back[:, None] + i).clamp(max=L - 1)
    vals = _decode(unpack(_bytes(codes)).view(codes.dtype), amax, c["block"], c["format"], torch.float32)
    got = vals.gather(2, at[:, None, :, None].expand(-1, h, -1, D)).transpose(1, 2).reshape(B, rows, h * D).to(out.dtype)
    keep = (i < n[:, None])[..., None]
    return torch.where(keep, got, out.view(B, rows, h * D)).view(B * rows, h * D)


def _plain_attn(s):
    c = s["case"]
    B, rows, H, h, D = c["B"], c["rows"], c["heads"], c["n_kv"], c["dim"]
    L, group = s["k"].shape[2], H // h
    k = _decode(_unpack_k(_bytes(s["k"])).view(s["k"].dtype), s["ka"], c["block"], c["format"], torch.float32)
    q = s["q"].float().view(B, rows, h, group, D).permute(0, 2, 1, 3, 4).reshape(B, h, rows * group, D)
    z = (q @ k.transpose(2, 3)) * s["scale"]
    del k
    p = torch.arange(L, device=z.device)
    i = torch.arange(rows, device=z.device).repeat_interleave(group)
    seen = (p >= s["first"][:, None, None]) & (p <= s["lens"][:, None, None] + i[:, None])  # [B, rows group, L]
    z = z.masked_fill(~seen[:, None], -math.inf)
    m = z.amax(3, keepdim=True)
    e = torch.exp(z - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    total = e.sum(3, keepdim=True)
    v = _decode(_unpack_v(_bytes(s["v"])).view(s["v"].dtype), s["va"], c["block"], c["format"], torch.float32)
    o = (e / torch.where(total > 0, total, torch.ones_like(total))) @ v
    return o.view(B, h, rows, group, D).permute(0, 2, 1, 3, 4).reshape(B * rows, H * D).bfloat16()


def _plain_logprob(s):
    c = s["case"]
    n, V = c["top"], c["V"]
    z = s["h"].float() @ s["lm"].float().T
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    entropy = torch.log(total)[:, 0] - (e * (z - m)).sum(1) / total[:, 0]
    # the order of close alternatives in 64 bits: candidates in 32, decided on their exact products
    few = min(V, n + 16)
    ids = torch.topk(z, few, dim=1).indices.sort(1).values
    z64 = (s["lm"][ids].double() @ s["h"].double()[:, :, None])[..., 0]
    order = torch.sort(z64, dim=1, descending=True, stable=True).indices[:, :n]
    t64 = (s["h"].double() * s["lm"][s["tok"].long()].double()).sum(1)
    return {"logprob": (t64 - lse.double()).float(), "entropy": entropy, "ids": ids.gather(1, order).int(),
            "top": (z64.gather(1, order) - lse.double()[:, None]).float()}


# ------------------------------------------------------------------ 64 bits
def _grid64(x, fmt):
    """The nearest code value to x, ties to even."""
    if fmt == "int8":
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _codes64(codes, packed_v):
    """[h, L, D] code values of one sequence, read off the documented places."""
    h, L, D = codes.shape
    p, d = torch.arange(L, device=codes.device)[:, None], torch.arange(D, device=codes.device)
    if packed_v:
        at = p // 16 * 16 * D + d // 4 * 64 + p % 16 // 4 * 16 + d % 4 * 4 + p % 4
    else:
        at = p // 16 * 16 * D + d // 64 * 1024 + p % 16 * 64 + d % 64
    return _bytes(codes).reshape(h, L * D)[:, at].view(codes.dtype).double()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "logprob":
        lm, parts = s["lm"].double(), []
        for i in range(0, c["R"], 512):
            z = s["h"][i:i + 512].double() @ lm.T
            lp = z - torch.logsumexp(z, 1, keepdim=True)
            p = lp.exp()
            parts.append((lp.gather(1, s["tok"][i:i + 512, None].long())[:, 0], -(p * lp).sum(1), torch.topk(lp, c["top"], dim=1).values))
        return {"logprob": torch.cat([x[0] for x in parts]), "entropy": torch.cat([x[1] for x in parts]), "ids": None,
                "top": torch.cat([x[2] for x in parts])}
    B, h, D, block, fmt, rows, Q = c["B"], c["n_kv"], c["dim"], c["block"], c["format"], c["rows"], Q_OF[c["format"]]
    if c["op"] == "attn":
        lens, first, _ = _attn_lens(c)
        group, o = c["heads"] // h, []
        for b in range(B):
            lo, hi = first[b], lens[b] + rows
            kb, vb = (_codes64(s[x][b], x == "v")[:, lo:hi] * s[x + "a"][b].double().repeat_interleave(block, 1)[:, lo:hi, None] / Q
                      for x in ("k", "v"))
            q = s["q"].view(B, rows, h, group, D)[b].double().permute(1, 0, 2, 3).reshape(h, rows * group, D)
            z = (q @ kb.transpose(1, 2)) * s["scale"]
            last = lens[b] + torch.arange(rows, device=DEV).repeat_interleave(group)
            z = torch.where(torch.arange(lo, hi, device=DEV) <= last[:, None], z, -math.inf)
            o.append((torch.softmax(z, 2) @ vb).view(h, rows, group, D).transpose(0, 1).reshape(rows, -1))
        return torch.cat(o)
    pos, n, _ = _row_counts(c)
    out = {}
    for x, part in (("k", 1), ("v", 2)):
        got = torch.zeros(B, s["rows_back"], h * D, dtype=torch.float64, device=DEV)
        amax = s[x + "a"].double()
        for b in range(B):
            codes = _codes64(s[x][b], x == "v")
            lo, hi = (int(s["back"][b]), int(s["back"][b]) + int(s["n_back"][b]))
            if c["op"] == "write":
                rows_b = s["qkv"].view(B, rows, 3, h, D)[b, :n[b], part].double().transpose(0, 1)
                for k in range(pos[b] // block, (pos[b] + n[b] - 1) // block + 1):
                    p0, p1 = max(k * block, pos[b]), min((k + 1) * block, pos[b] + n[b])
                    part_b = rows_b[:, p0 - pos[b]:p1 - pos[b]]
                    was = amax[b, :, k].clone() if p0 > k * block else torch.zeros(h, dtype=torch.float64, device=DEV)
                    now = torch.maximum(was, part_b.abs().amax((1, 2)))
                    codes[:, k * block:p0] = _grid64(codes[:, k * block:p0] * was[:, None, None] / now[:, None, None], fmt)  # exact at ties
                    codes[:, p0:p1] = _grid64(part_b * Q / now[:, None, None], fmt)
                    amax[b, :, k] = now
            got[b, :hi - lo] = (codes[:, lo:hi] * (amax[b].repeat_interleave(block, 1)[:, lo:hi, None] / Q)).transpose(0, 1).reshape(hi - lo, h * D)
        out[x] = got.view(-1, h * D)
        if c["op"] == "write":
            out[x + "_amax"] = amax
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "logprob":
        R, H, V = c["R"], c["H"], c["V"]
        return {"bytes": 2 * V * H + 2 * R * H + R * (12 + 8 * c["top"]), "flops": 2 * R * H * V}
    B, h, D, block, rows = c["B"], c["n_kv"], c["dim"], c["block"], c["rows"]
    if c["op"] == "attn":
        lens, first, _ = _attn_lens(c)
        seen = sum(n + rows - f for n, f in zip(lens, first))
        per = sum((n + rows - 1) // block - f // block + 1 for n, f in zip(lens, first))
        return {"bytes": 2 * h * (seen * D + 4 * per) + 4 * B * rows * c["heads"] * D, "flops": 4 * rows * c["heads"] * D * seen}
    pos, n, _ = _row_counts(c)
    wide = 2 if c["back"] == "bf16" else 4
    # keys and values: codes read, values written
    back = [(p % block if c["op"] == "write" else 0) + m for p, m in zip(pos, n)]
    total = 2 * h * D * sum(back) * (1 + wide)
    if c["op"] == "write":  # bf16 rows read, codes written
        total += 2 * h * D * sum(n) * 3
    return {"bytes": total, "flops": 4 * h * D * sum(back)}
