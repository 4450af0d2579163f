"""What the attention operators are measured on: writing keys and values to a
paged 4-bit cache, reading them back, attention over that cache, and attention
over a packed prompt.

`run` computes one pass in plain torch operations, or, where `own` is true,
through the public entry points of block_diffusion_moe_gb300.clover. Both take
what `prepare` makes from the seed."""
import math
import random

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # between code i and i + 1; a tie goes to the even code


def listed():
    return [
        # one new token of a conversation, written behind 999 others
        dict(name="write_token", op="write", seqs=1, new=1, before=999, ragged=False, pick=0, q_heads=16, kv_heads=2,
             dim=128, page=32, type="bf16"),
        # the prompts of five requests at once
        dict(name="write_prompt", op="write", seqs=5, new=4096, before=0, ragged=True, pick=1, q_heads=32, kv_heads=8,
             dim=128, page=64, type="bf16"),
        # short prefixes of a few requests, read back for a pass over the rest of their prompts
        dict(name="read_short", op="read", seqs=7, new=300, before=0, ragged=True, pick=2, q_heads=16, kv_heads=4, dim=64,
             page=16, type="bf16"),
        # a whole context of 131,072 tokens
        dict(name="read_long", op="read", seqs=1, new=131072, before=0, ragged=False, pick=0, q_heads=16, kv_heads=2,
             dim=128, page=64, type="bf16"),
        # one token of one conversation: what a single decoding step waits for
        dict(name="cached_token", op="cached", seqs=1, new=1, before=1020, ragged=False, pick=0, q_heads=16, kv_heads=2,
             dim=128, page=32, block=1, lse=False),
        # a serving batch of single tokens over contexts of different lengths
        dict(name="cached_batch", op="cached", seqs=64, new=1, before=16383, ragged=True, pick=3, q_heads=32, kv_heads=8,
             dim=128, page=64, block=1, lse=False),
        # a 32-position block being denoised over a long context: every position sees the whole block
        dict(name="cached_block", op="cached", seqs=1, new=32, before=131040, ragged=False, pick=0, q_heads=16, kv_heads=2,
             dim=128, page=64, block=0, lse=False),
        # the causal pass over eight finished blocks of requests of different lengths
        dict(name="cached_verify", op="cached", seqs=8, new=32, before=8160, ragged=True, pick=4, q_heads=32, kv_heads=4,
             dim=64, page=16, block=1, lse=True),
        # many short prompts packed together
        dict(name="prompt_short", op="prompt", seqs=40, new=200, before=0, ragged=True, pick=5, q_heads=16, kv_heads=2,
             dim=128, block=1, lse=False),
        # one long prompt
        dict(name="prompt_long", op="prompt", seqs=1, new=16384, before=0, ragged=False, pick=0, q_heads=16, kv_heads=2,
             dim=128, block=1, lse=False),
        # prompts cut into blocks of 32 that see themselves whole, as a block-diffusion model is prefilled
        dict(name="prompt_blocks", op="prompt", seqs=4, new=6000, before=0, ragged=True, pick=6, q_heads=32, kv_heads=8,
             dim=64, block=32, lse=False),
        # the next 1,000 tokens of two long prompts that are taken in pieces
        dict(name="prompt_chunk", op="prompt", seqs=2, new=1000, before=12000, ragged=False, pick=0, q_heads=16, kv_heads=2,
             dim=128, block=1, lse=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "cached", "cached", "prompt", "prompt"))
    kv_heads = rng.choice((1, 2, 3, 4, 8))
    c = dict(op=op, seqs=_log_int(rng, 1, 32), ragged=rng.random() < 0.7, pick=rng.randrange(1 << 30),
             kv_heads=kv_heads, q_heads=kv_heads * rng.choice((1, 2, 3, 4, 5, 7, 8)), dim=rng.choice((64, 128)))
    if op != "prompt":
        c["page"] = 16 * rng.choice((1, 2, 3, 4, 8))
    if op in ("write", "read"):
        return dict(c, new=_log_int(rng, 1, 4096), before=rng.choice((0, 0, _log_int(rng, 1, 4096))),
                    type=rng.choice(("bf16", "fp32")) if op == "write" else "bf16")
    c.update(block=rng.choice((0, 1, 1, 8, 32)), lse=rng.random() < 0.5)
    if op == "cached":
        c["q_heads"] *= rng.choice((1, 1, 2))
        return dict(c, new=rng.choice((1, 1, _log_int(rng, 2, 32))), before=_log_int(rng, 1, 16000))
    new = _log_int(rng, 1, 4096)
    return dict(c, seqs=min(c["seqs"], max(1, 8192 // new)), q_heads=kv_heads * rng.randint(1, 32 // kv_heads), new=new,
                before=rng.choice((0, 0, _log_int(rng, 1, 4096))))


def _lengths(case):
    """New tokens and whole length of each sequence."""
    rng = random.Random(case["pick"])
    new, length = [], []
    for _ in range(case["seqs"]):
        n, b = case["new"], case["before"]
        if case["ragged"]:
            n, b = _log_int(rng, max(1, n / 8), n), rng.randint(0, b)
        new.append(n)
        length.append(n + b)
    return new, length


# ------------------------------------------------------------------- inputs
#
# A page of the cache holds, for each head, its tokens in sixteens: 16 rows of
# key codes (two to a byte, the even element in the low half), 16 rows of key
# scales (e4m3, one for 16 elements), and the same of the values.


def _scale_of(y):
    """y fp32 [..., 16] -> the block scale: a sixth of the largest magnitude, as the e4m3 value nearest to it."""
    return (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()


def _codes_of(y, s):
    """The nearest e2m1 code of y / s (ties to the even code): |y| against border * s, both exact in fp32."""
    a = y.abs()
    code = torch.zeros(y.shape, dtype=torch.uint8, device=y.device)
    for i, b in enumerate(BORDERS):
        code += (a > b * s) if i % 2 == 0 else (a >= b * s) & (s > 0)
    return code, y < 0


def _pack(x):
    """fp32 [tokens, heads, dim] -> codes [tokens, heads, dim / 2] and scale bytes [tokens, heads, dim / 16]."""
    y = x.view(*x.shape[:2], -1, 16)
    s = _scale_of(y)
    code, neg = _codes_of(y, s[..., None])
    code = (code + 8 * neg.to(torch.uint8)).view(x.shape)
    return code[..., 0::2] + 16 * code[..., 1::2], s.to(torch.float8_e4m3fn).view(torch.uint8)


def _rows_of(tokens, g, heads, dim, outliers):
    """Rows such as keys and values are: a few channels of every head larger than the others."""
    x = torch.randn((tokens, heads, dim), generator=g, device=DEV)
    return x * torch.where(torch.rand((heads, dim), generator=g, device=DEV) < 0.03, outliers, 1.0)


def _parts(pages, dim):
    """Views of a pool [pages, heads, sixteens, bytes]: key codes, key scales, value codes, value scales, each
    [pages, heads, sixteens, 16, bytes of a row]."""
    sizes = (8 * dim, dim, 8 * dim, dim)
    return [p.unflatten(-1, (16, -1)) for p in pages.split(sizes, -1)]


def _places(table, length, page, lo=0):
    """(page, sixteen in the page, row in the sixteen) of positions lo .. length - 1 of one sequence."""
    i = torch.arange(lo, length, device=table.device)
    return table[i // page].long(), i % page // 16, i % 16


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    new, length = _lengths(case)
    H, Hq, D = case["kv_heads"], case["q_heads"], case["dim"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    T = at[-1]
    s = dict(case=case, new=new, length=length, at=at, offsets=ints(at), lens=ints(length), ws=None)
    if case["op"] == "prompt":
        s["k_at"] = [0]
        for n in length:
            s["k_at"].append(s["k_at"][-1] + n)
        s["k_offsets"] = s["offsets"] if new == length else ints(s["k_at"])
        Tk = s["k_at"][-1]
        if T == Tk:  # as one projection gives them, side by side
            qkv = torch.randn((T, Hq + 2 * H, D), generator=g, device=DEV)
            qkv[:, Hq:Hq + H] = _rows_of(T, g, H, D, 3.0)
            s["q"], s["k"], s["v"] = qkv.bfloat16().split((Hq, H, H), 1)
        else:
            s["q"] = torch.randn((T, Hq, D), generator=g, device=DEV).bfloat16()
            s["k"] = _rows_of(Tk, g, H, D, 3.0).bfloat16()
            s["v"] = torch.randn((Tk, H, D), generator=g, device=DEV).bfloat16()
        return s
    page = case["page"]
    used = [-(-n // page) for n in length]
    pool = sum(used) + 3
    free = torch.randperm(pool, generator=g, device=DEV).int()
    table = torch.full((case["seqs"], max(used)), -1, dtype=torch.int32, device=DEV)
    n = 0
    for i, u in enumerate(used):
        table[i, :u] = free[n:n + u]
        n += u
    s["table"] = table
    # what no token of a sequence lies in holds anything
    s["pages"] = torch.randint(0, 256, (pool, H, page // 16, 18 * D), generator=g, device=DEV, dtype=torch.uint8)
    if case["op"] == "write":
        s["k"], s["v"] = _rows_of(T, g, H, D, 8.0), _rows_of(T, g, H, D, 2.0)
        if case["type"] == "bf16":
            s["k"], s["v"] = s["k"].bfloat16(), s["v"].bfloat16()
        return s
    kc, ks, vc, vs = _parts(s["pages"], D)
    for i, L in enumerate(length):
        for lo in range(0, L, 16384):
            p, c, r = _places(table[i], min(L, lo + 16384), page, lo)
            kc[p, :, c, r], ks[p, :, c, r] = _pack(_rows_of(p.numel(), g, H, D, 3.0))
            vc[p, :, c, r], vs[p, :, c, r] = _pack(_rows_of(p.numel(), g, H, D, 1.0))
    if case["op"] == "cached":
        s["q"] = torch.randn((T, Hq, D), generator=g, device=DEV).bfloat16()
    return s


# -------------------------------------------------------------- plain forms


def _plain_write(s):
    out = []
    for x in (s["k"], s["v"]):
        y = x.float().view(*x.shape[:2], -1, 16)
        v = _scale_of(y)[..., None]
        code, neg = _codes_of(y, v)
        value = torch.tensor(E2M1, device=DEV)[code.int()] * v
        out.append(torch.where(neg, -value, value).view(x.shape).bfloat16())
    return tuple(out)


def _cached_rows(s, i, lo=0):
    """Keys and values of positions lo .. of sequence i, fp32 [tokens, heads, dim]."""
    D = s["case"]["dim"]
    p, c, r = _places(s["table"][i], s["length"][i], s["case"]["page"], lo)
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    kc, ks, vc, vs = (t[p, :, c, r] for t in _parts(s["pages"], D))
    out = []
    for codes, scales in ((kc, ks), (vc, vs)):
        q = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
        sc = scales.contiguous().view(torch.float8_e4m3fn).float()
        out.append((q.view(*sc.shape, 16) * sc[..., None]).view(q.shape))
    return out


def _plain_read(s):
    parts = [_cached_rows(s, i, L - n) for i, (n, L) in enumerate(zip(s["new"], s["length"]))]
    return tuple(torch.cat([p[j] for p in parts]).bfloat16() for j in (0, 1))


def _attend(q, k, v, block):
    """q [n, Hq, D], k and v [L, H, D] in fp32 -> out [n, Hq, D], lse [n, Hq]; the queries are the last n positions. A
    query sees the positions below the end of its own block (block 0: all of them)."""
    n, Hq, D = q.shape
    L, H, _ = k.shape
    G = Hq // H
    out, lse = torch.empty_like(q), torch.empty((n, Hq), device=q.device)
    kt, vt = k.permute(1, 2, 0), v.permute(1, 0, 2)
    step = max(1, (1 << 29) // (Hq * L))
    for lo in range(0, n, step):
        qi = q[lo:lo + step]
        m = qi.shape[0]
        x = torch.matmul(qi.view(m, H, G, D).permute(1, 0, 2, 3).reshape(H, m * G, D), kt) * D ** -0.5
        x = x.view(H, m, G, L)
        if block:
            pos = torch.arange(L - n + lo, L - n + lo + m, device=q.device)
            limit = (pos // block + 1) * block
            x = x.masked_fill_((torch.arange(L, device=q.device) >= limit[:, None])[None, :, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        e = x.sub_(top).exp_()
        total = e.sum(-1, keepdim=True)
        y = torch.matmul(e.view(H, m * G, L), vt).view(H, m, G, D) / total
        out[lo:lo + m] = y.permute(1, 0, 2, 3).reshape(m, Hq, D)
        lse[lo:lo + m] = (top + total.log())[..., 0].permute(1, 0, 2).reshape(m, Hq)
    return out, lse


def _plain_attention(s):
    c, outs, lses = s["case"], [], []
    for i in range(c["seqs"]):
        if c["op"] == "cached":
            k, v = _cached_rows(s, i)
        else:
            k, v = (s[t][s["k_at"][i]:s["k_at"][i + 1]].float() for t in "kv")
        o, lse = _attend(s["q"][s["at"][i]:s["at"][i + 1]].float(), k, v, c["block"])
        outs.append(o.bfloat16())
        lses.append(lse)
    out = torch.cat(outs)
    return (out, torch.cat(lses)) if c["lse"] else out


# ------------------------------------------------------- the framework's calls


def _own(s):
    from block_diffusion_moe_gb300 import clover

    c = s["case"]
    op = c["op"]
    if op != "prompt" and "cache" not in s:
        s["cache"] = clover.KvCache(s["pages"])
    if op == "write":
        clover.kv_write(s["cache"], s["k"], s["v"], s["offsets"], s["lens"], s["table"])
    if op in ("write", "read"):
        return clover.kv_read(s["cache"], s["offsets"], s["lens"], s["table"], s["at"][-1])
    T, seqs, heads = s["at"][-1], c["seqs"], c["q_heads"]
    if op == "cached":
        if s["ws"] is None:
            s["ws"] = clover.workspace(clover.kv_attention_workspace_bytes(s["cache"], T, heads, *s["table"].shape))
        return clover.kv_attention(s["q"], s["cache"], s["offsets"], s["lens"], s["table"], block=c["block"], lse=c["lse"],
                                   ws=s["ws"])
    if s["ws"] is None:
        s["ws"] = clover.workspace(clover.prompt_attention_workspace_bytes(T, s["k_at"][-1], seqs, heads, c["kv_heads"],
                                                                           c["dim"]))
    return clover.prompt_attention(s["q"], s["k"], s["v"], s["offsets"], s["k_offsets"], block=c["block"], lse=c["lse"],
                                   ws=s["ws"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"write": _plain_write, "read": _plain_read, "cached": _plain_attention, "prompt": _plain_attention}[op](state)


# ------------------------------------------------------------- work and exact


def _pairs(case):
    """Keys that the queries see, summed over the queries of one head."""
    new, length = _lengths(case)
    b = case["block"]
    if b == 0:
        return sum(n * L for n, L in zip(new, length))
    return sum(min(L, (p // b + 1) * b) for n, L in zip(new, length) for p in range(L - n, L))


def work(case):
    new, length = _lengths(case)
    T, L, H, Hq, D = sum(new), sum(length), case["kv_heads"], case["q_heads"], case["dim"]
    row = 9 * D // 8  # bytes of a cached key with its value: D codes of each, D / 16 scales of each
    if case["op"] == "write":
        # the values come back as bf16; the codes and scales between the two calls are not counted
        return dict(bytes=2 * T * H * D * ((2 if case["type"] == "bf16" else 4) + 2), flops=12 * T * H * D)
    if case["op"] == "read":
        return dict(bytes=T * H * (row + 4 * D), flops=2 * T * H * D)
    return dict(bytes=4 * T * Hq * D + L * H * (row if case["op"] == "cached" else 4 * D) + 4 * T * Hq * case["lse"],
                flops=4 * D * Hq * _pairs(case))


def _nearest(v, digits, least):
    """v >= 0 in fp64 to the nearest value of `digits` fraction bits and exponent at least `least`, ties to even."""
    e = (torch.frexp(v).exponent - 1).clamp(min=least)
    step = ((e - digits + 1023).long() << 52).view(torch.float64)
    return torch.round(v / step) * step


def _decoded64(s, i):
    """Keys and values of sequence i in fp64, from the bytes of its pages in the order of the table."""
    c = s["case"]
    page, D, L = c["page"], c["dim"], s["length"][i]
    raw = s["pages"][s["table"][i, : -(-L // page)].long()]          # [pages, heads, sixteens, bytes]
    raw = raw.permute(1, 0, 2, 3).reshape(c["kv_heads"], -1, 18 * D)  # [heads, sixteens, bytes]
    out = []
    for base in (0, 9 * D):
        codes = raw[..., base:base + 8 * D].reshape(c["kv_heads"], -1, D // 2)[:, :L]
        b = raw[..., base + 8 * D:base + 9 * D].reshape(c["kv_heads"], -1, D // 16)[:, :L].long()
        e, f = (b >> 3) & 15, (b & 7).double()
        scale = torch.where(e > 0, (1 + f / 8) * ((e - 7 + 1023) << 52).view(torch.float64), f * 2.0 ** -9)
        nib = torch.stack((codes & 15, codes >> 4), -1).flatten(2).long()
        mag = nib & 7
        val = torch.where(mag < 4, mag * 0.5, torch.where(mag < 6, mag.double() - 2.0, 2.0 * mag - 8.0))
        val = torch.where(nib > 7, -val, val)
        out.append((val.view(*scale.shape, 16) * scale[..., None]).view(nib.shape))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["dim"]
    if op == "write":
        out = []
        for x in (s["k"], s["v"]):
            y = x.double().view(*x.shape[:2], -1, 16)
            sc = _nearest(y.abs().amax(-1, keepdim=True) / 6.0, 3, -6).clamp(max=448.0)
            code = _nearest(y.abs() / sc.clamp(min=2.0 ** -300), 1, 0).clamp(max=6.0)
            out.append((torch.sign(y) * code * sc).view(x.shape))
        return tuple(out)
    if op == "read":
        both = [[t[:, L - n:].permute(1, 0, 2) for t in _decoded64(s, i)]
                for i, (n, L) in enumerate(zip(s["new"], s["length"]))]
        return tuple(torch.cat([b[j] for b in both]) for j in (0, 1))
    if work(case)["flops"] > 4e12:
        return None
    G = case["q_heads"] // case["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for i, (n, L) in enumerate(zip(s["new"], s["length"])):
        if op == "cached":
            k, v = _decoded64(s, i)
        else:
            k, v = (s[t][s["k_at"][i]:s["k_at"][i + 1]].permute(1, 0, 2).double() for t in "kv")
        rows = max(1, (1 << 28) // L)
        for lo in range(0, n, rows):
            at = slice(s["at"][i] + lo, s["at"][i] + min(n, lo + rows))
            p = L - n + torch.arange(lo, min(n, lo + rows), device=DEV)
            hidden = None
            if case["block"]:
                end = p - p % case["block"] + case["block"]
                hidden = end[:, None] <= torch.arange(L, device=DEV)
            for h in range(case["q_heads"]):
                z = s["q"][at, h].double() @ k[h // G].T / math.sqrt(D)
                if hidden is not None:
                    z[hidden] = -math.inf
                whole = torch.logsumexp(z, 1)
                lse[at, h] = whole
                out[at, h] = torch.exp(z - whole[:, None]) @ v[h // G]
    return (out, lse) if case["lse"] else out
