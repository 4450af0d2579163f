"""What the routed-expert operators are measured on: expert routing, microscaled
4-bit quantisation, the grouped 4-bit product and the weighted combine.

`run` computes one pass in plain torch operations, or, where `own` is true,
through the public entry points of block_diffusion_moe_gb300.clover. Both take
what `prepare` makes from the seed."""
import math

import torch

own = False

DEV = "cuda"
FLT_MAX = torch.finfo(torch.float32).max
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # between code i and i + 1; a tie goes to the even code


def listed():
    return [
        # one token of the 256-expert top-8 layer: what a single-token step waits for
        dict(name="route_token", op="route", M=1, E=256, K=8, score="softmax", bias=False, groups=1, top_groups=1,
             rank=1, renorm=True, scale=1.0, type="fp32", padded=0.0),
        # an odd batch of eight blocks and a bit, bf16 logits, a Zipf-like balance bias
        dict(name="route_batch", op="route", M=257, E=256, K=8, score="softmax", bias=True, groups=1, top_groups=1,
             rank=1, renorm=True, scale=1.0, type="bf16", padded=0.0),
        # a long prompt batch with padding rows, sigmoid scores, grouped selection
        dict(name="route_prompt", op="route", M=32768, E=256, K=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             rank=2, renorm=True, scale=2.5, type="fp32", padded=0.05),
        # one token's hidden row, copied to its eight experts and quantised
        dict(name="quantize_token", op="quantize", format="nv", mats=1, tokens=1, K=8, E=256, cols=2048, type="bf16",
             grouped=True),
        # a prompt's hidden rows gathered into expert order
        dict(name="quantize_prompt", op="quantize", format="mx", mats=1, tokens=8192, K=8, E=256, cols=2048,
             type="bf16", grouped=True),
        # the gate/up matrices of 64 experts, quantised once at load time
        dict(name="quantize_experts", op="quantize", format="nv", mats=64, tokens=1024, K=1, E=1, cols=2048,
             type="bf16", grouped=False),
        # one token through the down matrices of its eight experts
        dict(name="product_token", op="product", format="mx", tokens=1, K=8, E=256, N=2048, cols=512, swiglu=False),
        # a 32-position block through gate/up with SwiGLU: the denoising step's product
        dict(name="product_block", op="product", format="nv", tokens=32, K=8, E=256, N=1024, cols=2048, swiglu=True),
        # a prompt of 8,192 tokens through gate/up with SwiGLU
        dict(name="product_prompt", op="product", format="nv", tokens=8192, K=8, E=256, N=1024, cols=2048,
             swiglu=True),
        # one square matrix without groups: the rate of the product itself
        dict(name="product_dense", op="product", format="nv", tokens=8192, K=1, E=1, N=8192, cols=8192, swiglu=False),
        # one token's eight expert rows joined with the shared expert and the residual
        dict(name="combine_token", op="combine", M=1, K=8, H=2048, shared=True, padded=0.0),
        # the same for a prompt batch with padding rows
        dict(name="combine_prompt", op="combine", M=16384, K=8, H=2048, shared=True, padded=0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "quantize", "product", "combine"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * rng.randint(max(1, 8 // groups), 256 // groups)
        top_groups = rng.randint(1, groups)
        K = rng.randint(1, min(16, E))
        return dict(op=op, M=_log_int(rng, 1, 32768), E=E, K=K, score=rng.choice(("softmax", "sigmoid")),
                    bias=rng.random() < 0.6, groups=groups, top_groups=top_groups, rank=rng.choice((1, 2)),
                    renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)), type=rng.choice(("fp32", "bf16")),
                    padded=rng.choice((0.0, 0.1)))
    if op == "quantize":
        grouped = rng.random() < 0.6
        return dict(op=op, format=rng.choice(("nv", "mx")), mats=1 if grouped else rng.randint(1, 9),
                    tokens=_log_int(rng, 1, 4096), K=rng.randint(1, 8) if grouped else 1,
                    E=rng.randint(8, 256) if grouped else 1, cols=64 * _log_int(rng, 1, 40),
                    type=rng.choice(("bf16", "fp32")), grouped=grouped)
    if op == "product":
        E = rng.choice((1, 1, 8, 60, 128, 256))
        swiglu = rng.random() < 0.5
        cols = 64 * _log_int(rng, 1, 40)
        most = min(2500, (1 << 29) // (E * cols))
        N = 2 * _log_int(rng, 16, most // 4) if swiglu else _log_int(rng, 16, most)
        return dict(op=op, format=rng.choice(("nv", "mx")), tokens=_log_int(rng, 1, 4096),
                    K=rng.randint(1, min(8, E)), E=E, N=N, cols=cols, swiglu=swiglu)
    return dict(op=op, M=_log_int(rng, 1, 8192), K=rng.randint(1, 8), H=8 * _log_int(rng, 8, 500),
                shared=rng.random() < 0.5, padded=rng.choice((0.0, 0.1)))


# ------------------------------------------------------------------- inputs


def _grouping(idx, E):
    """Slots (token * K + k) in expert order, their offsets by expert and each slot's place; -1 marks no expert."""
    n = idx.numel()
    flat = idx.reshape(-1).long()
    key = torch.where(flat >= 0, flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    offsets[1:] = torch.cumsum(counts[:E], 0)
    taken = key[order] < E
    rows = torch.where(taken, order, -1)
    place = torch.arange(n, device=idx.device)
    pos = torch.empty_like(flat)
    pos[order] = torch.where(taken, place, -1)
    return offsets.int(), rows.int(), pos.int().view(idx.shape)


def _choices(M, K, E, g, padded=0.0):
    """K different experts for each token, some experts far more popular than others; padding rows choose none."""
    taste = torch.randn((M, E), generator=g, device=DEV) + 0.5 * torch.randn((1, E), generator=g, device=DEV)
    idx = torch.topk(taste, K, dim=1).indices.int()
    if padded:
        idx[torch.rand(M, generator=g, device=DEV) < padded] = -1
    return idx


def _power(e):
    """2^e in fp32 for whole e in [-126, 127], from its bits."""
    return ((e + 127).int() << 23).view(torch.float32)


def _scale_of(y, fmt):
    """y fp32 [..., blocks, block] -> the block scale, as the fp32 value it stands for."""
    amax = y.abs().amax(-1)
    if fmt == "nv":
        return (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    _, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1
    return torch.where(amax > 0, _power((e - 3).clamp(-126, 127)), 0.0)


def _codes_of(y, s):
    """The nearest e2m1 code of y / s (ties to the even code): |y| against border * s, both exact in fp32."""
    a = y.abs()
    code = torch.zeros(y.shape, dtype=torch.uint8, device=y.device)
    for i, b in enumerate(BORDERS):
        code += (a > b * s) if i % 2 == 0 else (a >= b * s) & (s > 0)
    return code, y < 0


def _tiled(sb):
    """Scale bytes [mats, rows, blocks] -> tiles of 128 rows x 4 blocks, byte (r % 32) * 16 + (r / 32) * 4 + b."""
    n, rows, nb = sb.shape
    sb = torch.nn.functional.pad(sb, (0, -nb % 4, 0, -rows % 128))
    return sb.view(n, sb.shape[1] // 128, 4, 32, sb.shape[2] // 4, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(-1)


def _untiled(tiles, n, rows, nb):
    t, c = -(-rows // 128), -(-nb // 4)
    sb = tiles.view(n, t, c, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, t * 128, c * 4)
    return sb[:, :rows, :nb]


def _padded_rows(offsets, n_rows):
    """Row of the scale tiles that belongs to each grouped row: every group begins a new tile of 128 rows."""
    off = offsets.long()
    i = torch.arange(n_rows, device=offsets.device)
    g = (torch.searchsorted(off, i, right=True) - 1).clamp(0, off.numel() - 2)
    return (off[g] // 128 + g) * 128 + (i - off[g]), g


def _pack(y, fmt, offsets=None):
    """fp32 [mats, rows, cols] -> packed codes [mats, rows, cols / 2] and tiled scale bytes."""
    n, rows, cols = y.shape
    block = 16 if fmt == "nv" else 32
    yb = y.view(n, rows, cols // block, block)
    s = _scale_of(yb, fmt)
    code, neg = _codes_of(yb, s[..., None])
    code = (code + 8 * neg.to(torch.uint8)).view(n, rows, cols)
    codes = code[..., 0::2] + 16 * code[..., 1::2]
    if fmt == "nv":
        sb = s.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        sb = torch.where(s > 0, torch.frexp(s)[1] + 126, 0).to(torch.uint8)
    if offsets is not None:
        at, _ = _padded_rows(offsets, rows)
        full = torch.zeros((1, (rows // 128 + offsets.numel() - 1) * 128, sb.shape[-1]), dtype=torch.uint8, device=y.device)
        full[0, at] = sb[0]
        sb = full
    return codes.contiguous(), _tiled(sb)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = dict(case=case, ws=None)
    if op == "route":
        M, E = case["M"], case["E"]
        x = 1.5 * torch.randn((M, E), generator=g, device=DEV) + 0.7 * torch.randn((1, E), generator=g, device=DEV)
        if case["padded"]:
            x[torch.rand(M, generator=g, device=DEV) < case["padded"]] = -math.inf
        s["logits"] = x if case["type"] == "fp32" else x.bfloat16()
        s["bias"] = 0.1 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
        n = M * case["K"]
        i32 = lambda *shape: torch.full(shape, -1, dtype=torch.int32, device=DEV)  # noqa: E731
        s["out"] = {"idx": i32(M, case["K"]), "w": torch.zeros((M, case["K"]), device=DEV), "offsets": i32(E + 1),
                    "rows": i32(n), "pos": i32(M, case["K"])}
    elif op == "quantize":
        rows, cols = case["tokens"], case["cols"]
        std = 1.0 if case["grouped"] else 0.02  # normed activations, expert weights
        x = std * torch.randn((case["mats"], rows, cols), generator=g, device=DEV)
        if case["grouped"]:  # a few features are far larger than the others
            x = x[0] * torch.where(torch.rand(cols, generator=g, device=DEV) < 0.01, 20.0, 1.0)
            idx = _choices(rows, case["K"], case["E"], g)
            s["offsets"], s["rows"], _ = _grouping(idx, case["E"])
        s["x"] = x.bfloat16() if case["type"] == "bf16" else x
        s["exp"] = 0 if case["grouped"] else -8
    elif op == "product":
        E, K, cols = case["E"], case["K"], case["cols"]
        idx = _choices(case["tokens"], K, E, g)
        s["offsets"], rows, _ = _grouping(idx, E)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        x = torch.randn((case["tokens"], cols), generator=g, device=DEV).bfloat16().float()
        s["a_codes"], s["a_scales"] = _pack(x[rows.long() // K][None], case["format"], s["offsets"])
        mats, n = (2 * E, case["N"] // 2) if case["swiglu"] else (E, case["N"])
        s["b_exp"] = -8 if case["format"] == "nv" else 0
        at, parts = max(1, (1 << 27) // (n * cols)), []
        for m in range(0, mats, at):
            w = 0.02 * torch.randn((min(at, mats - m), n, cols), generator=g, device=DEV)
            parts.append(_pack(w.bfloat16().float() * 2.0 ** -s["b_exp"], case["format"]))
        s["b_codes"] = torch.cat([p[0] for p in parts]).view(mats, n, cols // 2)
        s["b_scales"] = torch.cat([p[1] for p in parts])
        s["lut"] = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    else:
        M, K, H = case["M"], case["K"], case["H"]
        idx = _choices(M, K, 256, g, case["padded"])
        _, _, s["pos"] = _grouping(idx, 256)
        s["y"] = torch.randn((M * K, H), generator=g, device=DEV).bfloat16()
        w = torch.rand((M, K), generator=g, device=DEV) + 0.05
        s["w"] = torch.where(s["pos"] >= 0, w / w.sum(1, keepdim=True), 0.0)
        s["x"] = 2.0 * torch.randn((M, H), generator=g, device=DEV)
        s["shared"] = torch.randn((M, H), generator=g, device=DEV).bfloat16() if case["shared"] else None
    return s


# -------------------------------------------------------------- plain forms


def _plain_route(s):
    c = s["case"]
    M, E, K, G = c["M"], c["E"], c["K"], c["groups"]
    x = s["logits"].double().clamp(max=FLT_MAX)
    live = x > -math.inf  # false for NaN too
    if c["score"] == "softmax":
        m = torch.where(live, x, -math.inf).amax(1, keepdim=True)
        e = torch.where(live, torch.exp(x - m), 0.0)
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    total = score if s["bias"] is None else score + s["bias"].double()
    key = torch.where(live, x if s["bias"] is None else total, -math.inf)
    if G > 1:
        if c["rank"] == 1:
            group = key.view(M, G, E // G).amax(2)
        else:
            two = torch.sort(torch.where(live, total, -math.inf).view(M, G, E // G), dim=2, descending=True).values[..., :2]
            group = two[..., 0] + torch.where(two[..., 1:] > -math.inf, two[..., 1:], 0.0).sum(2)
        best = torch.sort(group, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        kept = torch.zeros((M, G), dtype=torch.bool, device=x.device).scatter_(1, best, True)
        key = torch.where(kept.repeat_interleave(E // G, 1), key, -math.inf)
    top = torch.sort(key, dim=1, descending=True, stable=True)
    idx = torch.where(top.values[:, :K] > -math.inf, top.indices[:, :K], -1)
    w = torch.where(idx >= 0, score.gather(1, idx.clamp(min=0)), 0.0)
    if c["renorm"]:
        w = torch.where(idx >= 0, w / w.sum(1, keepdim=True), 0.0)
    offsets, rows, pos = _grouping(idx, E)
    return {"idx": idx.int(), "w": (w * c["scale"]).float(), "offsets": offsets, "rows": rows, "pos": pos}


def _plain_quantize(s):
    c = s["case"]
    x = s["x"]
    if c["grouped"]:
        x = x[s["rows"].long() // c["K"]]
    block = 16 if c["format"] == "nv" else 32
    y = (x.float() * 2.0 ** -s["exp"]).view(*x.shape[:-1], c["cols"] // block, block)
    v = _scale_of(y, c["format"])[..., None]
    code, neg = _codes_of(y, v)
    value = torch.tensor(E2M1, device=DEV)[code.int()] * v * 2.0 ** s["exp"]
    return torch.where(neg, -value, value).view(x.shape).bfloat16()


def _decoded(codes, sb, fmt, lut):
    """codes [..., rows, cols / 2], scale bytes [..., rows, blocks] -> fp32 [..., rows, cols]."""
    q = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    if fmt == "nv":
        sc = sb.contiguous().view(torch.float8_e4m3fn).to(lut.dtype)
    else:
        sc = (sb.int() << 23).view(torch.float32).to(lut.dtype)
    return (q.view(*sb.shape, -1) * sc[..., None]).view(q.shape)


def _product(s, lut):
    """The rows of each group padded to the longest group, one batched product, and the rows taken out again."""
    c = s["case"]
    E, cols, fmt = c["E"], c["cols"], c["format"]
    n_rows, nb = c["tokens"] * c["K"], cols // (16 if fmt == "nv" else 32)
    at, g = _padded_rows(s["offsets"], n_rows)
    a = _decoded(s["a_codes"][0], _untiled(s["a_scales"], 1, (n_rows // 128 + E) * 128, nb)[0, at], fmt, lut)
    mats, n, _ = s["b_codes"].shape
    b = _decoded(s["b_codes"], _untiled(s["b_scales"], mats, n, nb), fmt, lut).view(E, c["N"], cols)
    place = torch.arange(n_rows, device=a.device) - s["offsets"].long()[g]
    full = torch.zeros((E, s["most"], cols), dtype=lut.dtype, device=a.device)
    full[g, place] = a
    return torch.bmm(full, b.transpose(1, 2))[g, place] * 2.0 ** s["b_exp"]


def _plain_product(s):
    y = _product(s, s["lut"])
    if s["case"]["swiglu"]:
        gate, up = y.chunk(2, 1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.bfloat16()


def _plain_combine(s):
    rows = s["y"][s["pos"].clamp(min=0).long()].float()
    out = s["x"] + (rows * torch.where(s["pos"] >= 0, s["w"], 0.0)[..., None]).sum(1)
    return out if s["shared"] is None else out + s["shared"].float()


# ------------------------------------------------------- the framework's calls


def _own(s):
    from block_diffusion_moe_gb300 import clover

    c = s["case"]
    op = c["op"]
    if op == "route":
        if s["ws"] is None:
            s["routing"] = clover.make_routing(c["E"], c["K"], score=c["score"], n_groups=c["groups"],
                                               top_groups=c["top_groups"], group_rank=c["rank"],
                                               renormalise=c["renorm"], scale=c["scale"])
            s["ws"] = clover.workspace(clover.route_workspace_bytes(s["routing"], c["M"]))
        return clover.route(s["routing"], s["logits"], bias=s["bias"], ws=s["ws"], out=s["out"])
    if op == "quantize":
        fmt = clover.FP4_NV if c["format"] == "nv" else clover.FP4_MX
        if c["grouped"]:
            q = clover.quantize_fp4(s["x"], fmt, offsets=s["offsets"], src_rows=s["rows"], src_div=c["K"])
        else:
            q = clover.quantize_fp4(s["x"], fmt, scale_exp=s["exp"])
        return clover.dequantize_fp4(q)
    if op == "product":
        if s["ws"] is None:
            fmt = clover.FP4_NV if c["format"] == "nv" else clover.FP4_MX
            s["ws"] = clover.workspace(clover.fp4_product_workspace_bytes())
            s["a"] = clover.Fp4(fmt, s["a_codes"][0], s["a_scales"], offsets=s["offsets"])
            s["b"] = clover.Fp4(fmt, s["b_codes"], s["b_scales"], scale_exp=s["b_exp"])
        return clover.fp4_product(s["a"], s["b"], swiglu=c["swiglu"], ws=s["ws"])
    return clover.moe_combine(s["y"], s["pos"], s["w"], x=s["x"], shared=s["shared"])


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "quantize": _plain_quantize, "product": _plain_product,
            "combine": _plain_combine}[state["case"]["op"]](state)


# ------------------------------------------------------------- work and exact


def work(case):
    op = case["op"]
    if op == "route":
        M, E, K = case["M"], case["E"], case["K"]
        return dict(bytes=M * E * (4 if case["type"] == "fp32" else 2) + 16 * M * K + 4 * (E + 1), flops=8 * M * E)
    if op == "quantize":
        # the values come back as bf16; the codes and scales between the two calls are not counted
        size, src = (2 if case["type"] == "bf16" else 4), case["mats"] * case["tokens"] * case["cols"]
        return dict(bytes=src * size + src * case["K"] * 2, flops=6 * src * case["K"])
    if op == "product":
        rows, N, cols, E = case["tokens"] * case["K"], case["N"], case["cols"], case["E"]
        per = cols / 2 + cols / (16 if case["format"] == "nv" else 32)
        used = E * (1.0 - (1.0 - case["K"] / E) ** case["tokens"])  # groups that have rows, when chosen evenly
        return dict(bytes=rows * per + used * N * per + rows * (N // 2 if case["swiglu"] else N) * 2,
                    flops=2 * rows * N * cols)
    M, K, H = case["M"], case["K"], case["H"]
    return dict(bytes=M * K * H * 2 + M * H * (8 + 2 * case["shared"]) + 8 * M * K, flops=2 * M * K * H)


def _power64(e):
    return ((e + 1023).long() << 52).view(torch.float64)


def _round_to(v, digits, least):
    """v >= 0 in fp64 to the nearest value of `digits` fraction bits and exponent at least `least`, ties to even."""
    e = (torch.frexp(v).exponent - 1).clamp(min=least)
    step = _power64(e - digits)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        # the weights of the plain form's experts, from log-sum-exp and log-sigmoid in 64 bits
        x = s["logits"].double()
        idx = _plain_route(s)["idx"].long()
        if case["score"] == "softmax":
            log = x - torch.logsumexp(x, 1, keepdim=True)
        else:
            log = torch.where(x > 0, -torch.log1p(torch.exp(-x)), x - torch.log1p(torch.exp(x)))
        log = torch.where(idx >= 0, log.gather(1, idx.clamp(min=0)), -math.inf)
        if case["renorm"]:
            log = log - torch.logsumexp(log, 1, keepdim=True)
        w = torch.where(idx >= 0, torch.exp(log), 0.0) * case["scale"]
        return {"idx": None, "w": w, "offsets": None, "rows": None, "pos": None}
    if op == "quantize":
        x = s["x"].double()
        if case["grouped"]:
            x = x[s["rows"].long() // case["K"]]
        block = 16 if case["format"] == "nv" else 32
        y = (x * 2.0 ** -s["exp"]).view(*x.shape[:-1], -1, block)
        top = y.abs().amax(-1, keepdim=True)
        if case["format"] == "nv":
            sc = _round_to(top / 6.0, 3, -6).clamp(max=448.0)
        else:
            sc = _power64(torch.frexp(top).exponent - 3)
        q = _round_to(y.abs() / sc.clamp(min=2.0 ** -300), 1, 0).clamp(max=6.0)
        return (torch.sign(y) * q * sc * 2.0 ** s["exp"]).view(x.shape)
    if op == "product":
        if 2.0 * case["tokens"] * case["K"] * case["N"] * case["cols"] > 2e12:
            return None
        y = _product(s, s["lut"].double())
        if case["swiglu"]:
            gate, up = y.chunk(2, 1)
            y = gate * up * torch.sigmoid(gate)
        return y
    out = s["x"].double()
    for k in range(case["K"]):
        p = s["pos"][:, k].long()
        out = out + torch.where(p >= 0, s["w"][:, k].double(), 0.0)[:, None] * s["y"][p.clamp(min=0)].double()
    return out if s["shared"] is None else out + s["shared"].double()
