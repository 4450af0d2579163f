"""Expert routing, 4-bit quantisation and the weighted combine on the GPU
against the fp64 oracle (oracle/moe_ops.py). Every call goes through the C ABI.

Tolerances: u = 2^-24 is half a step of fp32 relative to a value. Indices,
groupings, codes and scales have to be equal."""
import numpy as np
import pytest
import torch

from block_diffusion_moe_gb300 import clover as C
from oracle import moe_ops as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _check_route(logits, r_kw, bias=None, out=None, ws=None):
    """logits: a tensor on the device. Compares every output with the oracle; returns the outputs."""
    M, E = logits.shape
    r = C.make_routing(E, **r_kw)
    got = C.route(r, logits, bias=bias, out=out, ws=ws)
    torch.cuda.synchronize()
    kw = {k: v for k, v in r_kw.items() if k != "top_k"}
    kw.setdefault("top_groups", kw.get("n_groups", 1))
    z = logits.float().cpu().numpy()
    ref = R.route(z, r_kw["top_k"], bias=None if bias is None else bias.cpu().numpy(), **kw)
    assert np.array_equal(got["idx"].cpu().numpy(), ref["idx"])
    assert np.array_equal(got["offsets"].cpu().numpy(), ref["offsets"])
    assert np.array_equal(got["pos"].cpu().numpy(), ref["pos"])
    n = int(ref["offsets"][-1])
    assert np.array_equal(got["rows"][:n].cpu().numpy(), ref["rows"])
    # an exponential is off by its argument's rounding (at most the range of the live logits, 2u each for the two
    # subtractions and the exponent) and 4u of its own; a sum of up to 512 terms in a tree of 16 + 5 adds 21u; the
    # quotient, the sigmoid's sum and the scale 4u
    live = z[np.isfinite(z)]
    span = min(float(live.max() - live.min()), 110.0) if live.size else 0.0
    tol = (2 * span + 60) * U
    w = got["w"].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(w - ref["w"]) <= tol * np.abs(ref["w"]) + 1e-37)
    return got


SHAPES = [  # M, E, K
    (1, 256, 8), (1, 1, 1), (2, 7, 7), (3, 32, 32), (9, 60, 6), (64, 64, 2), (65, 65, 3), (130, 128, 1), (257, 256, 8),
    (70, 384, 10), (33, 512, 32), (16, 256, 8), (256, 512, 4), (512, 256, 8), (513, 256, 8),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,K", SHAPES)
def test_route_shapes(M, E, K, score):
    g = _gen(M * 1000 + E)
    z = 2 * torch.randn(M, E, generator=g)
    _check_route(z.to(DEV), dict(top_k=K, score=score))
    b = 0.2 * torch.randn(E, generator=g)
    _check_route(z.to(DEV), dict(top_k=K, score=score, renormalise=False, scale=2.5), bias=b.to(DEV))
    _check_route(z.bfloat16().to(DEV), dict(top_k=K, score=score), bias=b.to(DEV))


@pytest.mark.parametrize("rank", [1, 2])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,top", [(256, 8, 4), (60, 4, 1), (64, 32, 5), (512, 2, 1), (24, 24, 9), (9, 3, 3), (8, 1, 1)])
def test_route_groups(E, G, top, score, with_bias, rank):
    g = _gen(E + G)
    z = 1.5 * torch.randn(40, E, generator=g)
    z[3] = -float("inf")
    z[5, : E // 2] = -float("inf")
    z[7, 1:] = float("nan")
    b = (0.3 * torch.randn(E, generator=g)).to(DEV) if with_bias else None
    _check_route(z.to(DEV), dict(top_k=min(6, E), score=score, n_groups=G, top_groups=top, group_rank=rank), bias=b)
    _check_route(z.bfloat16().to(DEV), dict(top_k=min(3, E), score=score, n_groups=G, top_groups=top, group_rank=rank), bias=b)


@pytest.mark.parametrize("M", [500, 2433, 2600, 20000])
def test_route_many_tokens(M):
    """Counts over several CTAs (2,433 tokens begin a larger tile per CTA), some tokens without an expert."""
    g = _gen(M)
    z = torch.randn(M, 40, generator=g) + 1.5 * torch.randn(1, 40, generator=g)
    z[torch.rand(M, generator=g) < 0.1] = -float("inf")
    b = (0.1 * torch.randn(40, generator=g)).to(DEV)
    _check_route(z.to(DEV), dict(top_k=4, score="sigmoid"), bias=b)


def test_route_ties_and_signed_zeros():
    z = torch.zeros(5, 96)
    z[1, ::2] = -0.0
    z[2] = 3.0
    z[3, 50:] = 1.0
    z[4] = -200.0  # every sigmoid is below the smallest float
    for score in ("softmax", "sigmoid"):
        _check_route(z.to(DEV), dict(top_k=8, score=score))
        _check_route(z.to(DEV), dict(top_k=8, score=score, n_groups=8, top_groups=3, group_rank=2))
        _check_route(z.to(DEV), dict(top_k=8, score=score), bias=torch.zeros(96, device=DEV))
        _check_route(z.to(DEV), dict(top_k=8, score=score, n_groups=8, top_groups=3, group_rank=1), bias=torch.ones(96, device=DEV))


@pytest.mark.parametrize("low", [False, True])
def test_route_scores_around_the_smallest_float(low):
    """Sigmoids on both sides of 2^-126 (logits of -87.3), or all below it, in more tokens than warps."""
    z = torch.empty(6000, 96).uniform_(-110.0 if low else -92.0, -88.0 if low else -84.0, generator=_gen(14))
    z[::7, 3] = 0.5
    z[1::7, ::2] = 90.0
    for kw in (dict(n_groups=6, top_groups=2, group_rank=2), dict(n_groups=8, top_groups=4, group_rank=1)):
        _check_route(z.to(DEV), dict(top_k=8, score="sigmoid", **kw))
        b = torch.zeros(96)
        b[10:20] = 1e-38
        _check_route(z.to(DEV), dict(top_k=8, score="sigmoid", **kw), bias=b.to(DEV))


def test_route_no_expert_left():
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[-inf] * 8, [nan] * 8, [-inf] * 7 + [1.0], [nan, 2.0] * 4, [inf] * 3 + [0.0] * 5,
                      [-3e38, 3e38, inf, -inf, nan, 0.0, 1.0, 2.0]])
    b = torch.tensor([0.0, 0.5, nan, -inf, 0.1, 0.2, 0.3, 0.4])
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = _check_route(z.to(DEV), dict(top_k=4, score=score, renormalise=renorm))
            assert got["idx"][0].tolist() == [-1] * 4 and got["w"][1].tolist() == [0.0] * 4
            _check_route(z.to(DEV), dict(top_k=4, score=score, renormalise=renorm), bias=b.to(DEV))
            _check_route(z.to(DEV), dict(top_k=4, score=score, n_groups=4, top_groups=2, group_rank=2), bias=b.to(DEV))
    _check_route(torch.full((200, 40), -inf, device=DEV), dict(top_k=4))


def test_route_infinite_biases():
    z = torch.randn(20, 96, generator=_gen(12))
    b = 0.1 * torch.randn(96, generator=_gen(13))
    b[5], b[60], b[7] = float("inf"), float("inf"), -float("inf")
    for score in ("softmax", "sigmoid"):
        _check_route(z.to(DEV), dict(top_k=4, score=score), bias=b.to(DEV))
        _check_route(z.to(DEV), dict(top_k=4, score=score, n_groups=6, top_groups=2, group_rank=2), bias=b.to(DEV))
        _check_route(z[:, :24].contiguous().to(DEV), dict(top_k=4, score=score, n_groups=3, top_groups=1, group_rank=1),
                     bias=b[:24].contiguous().to(DEV))


def test_route_keys_closer_than_fp32():
    """Keys that differ by about 1e-9: their order is that of the exact sums, which fp32 cannot tell."""
    rng = np.random.default_rng(5)
    M, E = 64, 64
    b = rng.normal(size=E).astype(np.float32) * np.float32(0.01)
    z = np.zeros((M, E), dtype=np.float32)
    for t in range(M):
        # aim each sigmoid at 0.6 - b, then round the logit: the keys end within some 1e-8 of 0.6
        p = 0.6 - b.astype(np.float64)
        z[t] = np.log(p / (1 - p)).astype(np.float32) + rng.integers(-1, 2, size=E).astype(np.float32) * np.float32(2.0 ** -25)
    s = 1 / (1 + np.exp(-z.astype(np.float64))) + b
    gaps = np.diff(np.sort(s, axis=1)[:, -9:], axis=1)
    assert gaps.max() < 1e-7 and np.median(gaps) > 1e-13  # closer than fp32's error, further than fp64's
    zt, bt = torch.from_numpy(z).to(DEV), torch.from_numpy(b).to(DEV)
    _check_route(zt, dict(top_k=8, score="sigmoid"), bias=bt)
    _check_route(zt, dict(top_k=8, score="sigmoid", n_groups=8, top_groups=4, group_rank=1), bias=bt)
    _check_route(zt, dict(top_k=8, score="sigmoid", n_groups=8, top_groups=4, group_rank=2), bias=bt)


def test_route_softmax_keys_closer_than_fp32():
    """Softmax scores with a bias each, aimed at one sum, the logits rounded and moved by a step: keys some 1e-9 apart,
    among scores that differ (so that an error of the softmax's sum could turn their order) and a few that do not."""
    rng = np.random.default_rng(8)
    M, E = 48, 64
    z = rng.normal(size=(M, E)).astype(np.float32)
    z[:, 1::16] = z[:, 0::16]
    b = np.zeros((M, E), dtype=np.float32)
    for t in range(M):
        p = np.exp(z[t].astype(np.float64))
        p /= p.sum()
        b[t] = (0.7 - p).astype(np.float32)  # off by up to 3e-8
        b[t, 1::16] = b[t, 0::16]
        for k in (dict(top_k=8), dict(top_k=3, n_groups=8, top_groups=2, group_rank=1),
                  dict(top_k=8, n_groups=4, top_groups=2, group_rank=2)):
            _check_route(torch.from_numpy(z[t:t + 1]).to(DEV), dict(k, score="softmax"), bias=torch.from_numpy(b[t]).to(DEV))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_strided_rows(dtype):
    z = torch.randn(50, 101, generator=_gen(3)).to(dtype).to(DEV)
    _check_route(z[:, 3:67], dict(top_k=5))
    _check_route(z[::2, 1:60], dict(top_k=5, score="sigmoid"))
    _check_route(z[:1, :64], dict(top_k=5))


def test_route_without_grouping_and_empty():
    z = torch.randn(70, 64, generator=_gen(4)).to(DEV)
    r = C.make_routing(64, 4)
    a, b = C.route(r, z), C.route(r, z, grouping=False)
    assert torch.equal(a["idx"], b["idx"]) and torch.equal(a["w"], b["w"]) and "pos" not in b
    e = C.route(r, z[:0])
    assert e["offsets"].tolist() == [0] * 65 and e["idx"].shape == (0, 4)


def test_route_leaves_places_behind_the_last():
    z = torch.randn(300, 32, generator=_gen(6)).to(DEV)
    z[::3] = -float("inf")
    r = C.make_routing(32, 2)
    out = C.route(r, z)
    out["rows"].fill_(-77)
    ws = torch.full((C.route_workspace_bytes(r, 300),), 0x5A, dtype=torch.uint8, device=DEV)  # its contents do not matter
    got = _check_route(z, dict(top_k=2), out=out, ws=ws)
    assert got["rows"][int(got["offsets"][-1]):].eq(-77).all() and int(got["offsets"][-1]) == 400


# --------------------------------------------------------------- quantisation


def _host_scales(q, n_tiles, blocks):
    return q.scales.cpu().numpy()[: n_tiles * -(-blocks // 4) * 512].reshape(n_tiles, -(-blocks // 4), 512)


def _check_codes(q, x_rows, fmt, scale_exp, scale_rows, n_tiles):
    """Codes and scale bytes of the listed rows against the oracle, bit for bit."""
    block = 16 if fmt == "nv" else 32
    codes, sb = R.quantize(x_rows, fmt, scale_exp)
    got = q.codes.reshape(-1, q.codes.shape[-1])[: len(codes)].cpu().numpy()
    assert np.array_equal(got, R.pack_codes(codes))
    tiles = _host_scales(q, n_tiles, codes.shape[1] // block)
    for i, sr in enumerate(scale_rows):
        for b in range(sb.shape[1]):
            assert tiles[R.scale_place(sr, b)] == sb[i, b], (i, b)
    return codes, sb


FMT = {"nv": C.FP4_NV, "mx": C.FP4_MX}


def _planted(rows, cols, seed):
    """Values on and next to every border, zeros, signed zeros, blocks of one value, tiny and huge blocks."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols)) * 2.0 ** rng.integers(-12, 12, size=(rows, 1))
    b = np.array([0, -0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 0.24902, 0.7539, -1.2578, 1.7421, -2.5156, 5.03])
    x[0, :16], x[0, 16:32] = b, -b[::-1]
    x[0, 32:64] = np.concatenate([b, b]) * 2.0 ** 7
    if rows > 1:
        x[1, :32] = 0.0
        x[1, 32:64] = 2.0 ** -30
    if rows > 2:
        x[2, :32] = 1e30 * rng.normal(size=32)
        x[2, 32:64] = 2.0 ** -6 * np.repeat(b, 2)
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("shape", [(1, 64), (3, 192), (2, 130, 64), (5, 7, 320), (3, 2112)])
def test_quantize_matrices(shape, fmt, dtype):
    x = torch.from_numpy(_planted(int(np.prod(shape[:-1])), shape[-1], 7)).to(dtype)
    rows, mats = shape[-2], shape[0] if len(shape) == 3 else 1
    padded = -(-rows // 128) * 128
    for exp in (0, -8, 5):
        q = C.quantize_fp4(x.view(shape).to(DEV), FMT[fmt], scale_exp=exp)
        flat = x.float().numpy()
        codes, sb = _check_codes(q, flat, fmt, exp, [m * padded + r for m in range(mats) for r in range(rows)],
                                 mats * padded // 128)
        back = C.dequantize_fp4(q)
        want = torch.from_numpy(R.dequantize(codes, sb, fmt, exp)).to(torch.bfloat16)
        assert torch.equal(back.cpu().reshape(want.shape), want)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_quantize_fp32_next_to_borders(fmt):
    """fp32 values one step to either side of border * scale land on their own side."""
    rng = np.random.default_rng(9)
    x = np.zeros((64, 64), dtype=np.float32)
    for r in range(64):
        s = np.float32(R.E4M3[rng.integers(30, 120)]) if fmt == "nv" else np.float32(2.0 ** rng.integers(-20, 20))
        v = (np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32)[rng.integers(0, 7, size=64)] * s)
        step = rng.integers(-1, 2, size=64)
        v = np.where(step < 0, np.nextafter(v, np.float32(0)), np.where(step > 0, np.nextafter(v, np.float32(1e30)), v))
        v[::16] = 6 * s
        x[r] = v * rng.choice([-1, 1], size=64)
    q = C.quantize_fp4(torch.from_numpy(x).to(DEV), FMT[fmt])
    _check_codes(q, x, fmt, 0, range(64), 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_quantize_non_finite_and_extreme(fmt, dtype):
    x = torch.randn(6, 128, generator=_gen(2))
    x[0, 5], x[1, 40], x[2, 100] = float("nan"), float("inf"), -float("inf")
    x[3] *= 2.0 ** 120
    x[4] *= 2.0 ** -126
    x[5] = 2.0 ** -133
    x = x.to(dtype)
    q = C.quantize_fp4(x.to(DEV), FMT[fmt])
    _check_codes(q, x.float().numpy(), fmt, 0, range(6), 1)
    back = C.dequantize_fp4(q).cpu()
    block = 16 if fmt == "nv" else 32
    assert back[0, :block].isnan().all() and not back[0, block:].isnan().any()
    assert back[1].isnan().sum() == block and back[2].isnan().sum() == block


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("tokens,K,E,cols", [(1, 8, 256, 128), (50, 3, 5, 192), (300, 2, 4, 64), (7, 1, 1, 64)])
def test_quantize_rows_in_expert_order(tokens, K, E, cols, fmt):
    """Rows gathered as route lists them; some tokens choose no expert, so the last rows stay as they were."""
    g = _gen(tokens)
    z = torch.randn(tokens, E, generator=g)
    if tokens > 4:
        z[1::4] = -float("inf")
    ref = C.route(C.make_routing(E, K), z.to(DEV))
    off = ref["offsets"].cpu().numpy()
    n = int(off[-1])
    x = torch.randn(tokens, cols, generator=g).bfloat16()
    out = C.quantize_fp4(x.to(DEV), FMT[fmt], offsets=ref["offsets"], src_rows=ref["rows"], src_div=K)
    out.codes.fill_(0xA5)
    q = C.quantize_fp4(x.to(DEV), FMT[fmt], offsets=ref["offsets"], src_rows=ref["rows"], src_div=K, out=out)
    rows = ref["rows"][:n].cpu().numpy()
    codes, sb = _check_codes(q, x.float().numpy()[rows // K], fmt, 0, [R.grouped_scale_row(i, off) for i in range(n)],
                             tokens * K // 128 + E)
    assert q.codes[n:].eq(0xA5).all()
    back = torch.full((tokens * K, cols), 9.0, dtype=torch.bfloat16, device=DEV)
    C.dequantize_fp4(q, out=back)
    assert torch.equal(back[:n].cpu(), torch.from_numpy(R.dequantize(codes, sb, fmt)).bfloat16())
    assert back[n:].eq(9.0).all()


def test_quantize_rows_bad_indices():
    """Offsets past the rows count as the nearer end, a source outside x as a row of zeros."""
    x = torch.randn(4, 64, generator=_gen(8)).bfloat16().to(DEV)
    src = torch.tensor([0, -5, 3, 4, 99, 2], dtype=torch.int32, device=DEV)
    off = torch.tensor([-3, 2, 2, 900], dtype=torch.int32, device=DEV)
    q = C.quantize_fp4(x, C.FP4_NV, offsets=off, src_rows=src)
    back = C.dequantize_fp4(q).cpu()
    good = C.dequantize_fp4(C.quantize_fp4(x, C.FP4_NV)).cpu()
    for i, s in enumerate((0, None, 3, None, None, 2)):
        assert torch.equal(back[i], good[s] if s is not None else torch.zeros(64, dtype=torch.bfloat16)), i
    C.quantize_fp4(x, C.FP4_MX, offsets=torch.tensor([3, 1, 0, 2], dtype=torch.int32, device=DEV), src_rows=src)
    torch.cuda.synchronize()


def test_quantized_parts_are_the_whole():
    """codes and scales as tensors make the same matrix again; an empty one has its shape."""
    x = torch.randn(3, 70, 192, generator=_gen(21)).to(DEV)
    q = C.quantize_fp4(x, C.FP4_MX, scale_exp=-3)
    assert q.codes.shape == (3, 70, 96) and q.scales.numel() == C.fp4_scale_bytes(C.FP4_MX, 3, 70, 192)
    again = C.Fp4(C.FP4_MX, q.codes.clone(), q.scales.clone(), scale_exp=-3)
    assert torch.equal(C.dequantize_fp4(again), C.dequantize_fp4(q))
    e = C.quantize_fp4(x[:, :0].contiguous())
    assert e.codes.shape == (3, 0, 96) and C.dequantize_fp4(e).shape == (3, 0, 192)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    e = C.quantize_fp4(x[0, :0], offsets=off)
    assert e.codes.shape == (0, 96) and e.scales.numel() == C.fp4_scale_bytes(C.FP4_NV, 1, 0, 192, 2)


def test_quantize_strided_rows():
    x = torch.randn(40, 256, generator=_gen(1)).bfloat16().to(DEV)
    for v in (x[:, 64:192], x[::3, :128], x[5:6, 128:]):
        a, b = C.quantize_fp4(v, C.FP4_NV), C.quantize_fp4(v.contiguous(), C.FP4_NV)
        assert torch.equal(a.codes, b.codes) and torch.equal(C.dequantize_fp4(a), C.dequantize_fp4(b))


def test_quantize_and_combine_past_2_31_elements():
    """Rows that begin past 2^31 elements and bytes are those of the same rows alone."""
    rows, cols = 263000, 8192
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[:64].normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    x[64:-64] = 0
    x[-64:].normal_(generator=torch.Generator(device=DEV).manual_seed(2))
    q = C.quantize_fp4(x, C.FP4_NV)
    back = C.dequantize_fp4(q)
    for part in (slice(0, 64), slice(rows - 64, rows)):
        assert torch.equal(back[part], C.dequantize_fp4(C.quantize_fp4(x[part], C.FP4_NV)))
    del back, q
    pos = torch.tensor([[rows - 1, 3], [0, rows - 2]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[1.0, 2.0], [0.5, -1.0]], device=DEV)
    near = torch.cat([x[:4], x[-2:]])
    small = torch.tensor([[5, 3], [0, 4]], dtype=torch.int32, device=DEV)
    assert torch.equal(C.moe_combine(x, pos, w), C.moe_combine(near, small, w))


# -------------------------------------------------------------------- combine


@pytest.mark.parametrize("M,K,H", [(1, 8, 2048), (5, 1, 8), (33, 3, 72), (7, 32, 256), (300, 8, 520), (2, 9, 2056)])
@pytest.mark.parametrize("with_x", [False, True])
@pytest.mark.parametrize("with_shared", [False, True])
def test_combine(M, K, H, with_x, with_shared):
    g = _gen(M + H)
    n = M * K
    y = torch.randn(n, H, generator=g).bfloat16()
    pos = torch.randperm(n, generator=g).view(M, K).int()
    pos[torch.rand(M, K, generator=g) < 0.2] = -1
    w = torch.randn(M, K, generator=g)
    x = torch.randn(M, H, generator=g) if with_x else None
    sh = torch.randn(M, H, generator=g).bfloat16() if with_shared else None
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    out = C.moe_combine(y.to(DEV), pos.to(DEV), w.to(DEV), x=dev(x), shared=dev(sh))
    yd = y.double().numpy()
    ref = R.combine(yd, pos.numpy(), w.numpy(), None if x is None else x.numpy(), None if sh is None else sh.double().numpy())
    mag = R.combine(np.abs(yd), pos.numpy(), np.abs(w.numpy()), None if x is None else np.abs(x.numpy()),
                    None if sh is None else np.abs(sh.double().numpy()))
    # K + 2 fused additions, each off by u of a partial sum that is at most the sum of the magnitudes
    assert np.all(np.abs(out.cpu().numpy() - ref) <= (K + 2) * U * mag)
    if with_x:
        xd = x.to(DEV)
        assert C.moe_combine(y.to(DEV), pos.to(DEV), w.to(DEV), x=xd, shared=dev(sh), out=xd) is xd
        assert torch.equal(xd, out)


def test_combine_skips_slots_whatever_they_hold():
    y = torch.ones(4, 64, dtype=torch.bfloat16, device=DEV)
    y[3] = float("nan")
    pos = torch.tensor([[0, -1], [4, 1], [-1, -1], [2, 1 << 30]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.5, float("nan")], [float("inf"), 2.0], [float("nan"), float("nan")], [1.0, float("inf")]], device=DEV)
    out = C.moe_combine(y, pos, w)
    assert out[:, 0].tolist() == [0.5, 2.0, 0.0, 1.0] and out.isfinite().all()
    z = C.moe_combine(y[:0], pos, w, x=torch.ones(4, 64, device=DEV))
    assert z.eq(1.0).all()


# ---------------------------------------------------------- use of the calls


def test_captured_and_replayed_on_another_stream():
    """Two graphs that share one workspace, replayed in turn, with new inputs in place."""
    r = C.make_routing(64, 4, score="sigmoid", n_groups=8, top_groups=4, group_rank=2)
    M = 700
    z = torch.randn(M, 64, device=DEV)
    b = 0.1 * torch.randn(64, device=DEV)
    x = torch.randn(M, 128, device=DEV).bfloat16()
    ws = C.workspace(C.route_workspace_bytes(r, M))
    side = torch.cuda.Stream()
    outs, graphs = [], []
    with torch.cuda.stream(side):
        for _ in range(2):
            o = C.route(r, z, bias=b, ws=ws)  # first calls outside the capture load the kernels
            q = C.quantize_fp4(x, C.FP4_NV, offsets=o["offsets"], src_rows=o["rows"], src_div=4)
            d = C.dequantize_fp4(q)
            c = C.moe_combine(d, o["pos"], o["w"])
            outs.append((o, q, d, c))
        torch.cuda.synchronize()
        for o, q, d, c in outs:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                C.route(r, z, bias=b, ws=ws, out=o)
                C.quantize_fp4(x, C.FP4_NV, offsets=o["offsets"], src_rows=o["rows"], src_div=4, out=q)
                C.dequantize_fp4(q, out=d)
                C.moe_combine(d, o["pos"], o["w"], out=c)
            graphs.append(gr)
        for seed in range(3):
            z.copy_(torch.randn(M, 64, generator=_gen(seed)))
            for gr in graphs:
                gr.replay()
            want = C.route(r, z, bias=b)
            side.synchronize()
            for o, q, d, c in outs:
                assert all(torch.equal(o[k], want[k]) for k in want)
                assert torch.equal(c, outs[0][3])
    assert outs[0][3].abs().sum() > 0


def test_wrappers_refuse():
    r = C.make_routing(64, 4)
    z = torch.randn(8, 64, device=DEV)
    y = torch.randn(32, 64, device=DEV).bfloat16()
    pos = torch.zeros(8, 4, dtype=torch.int32, device=DEV)
    w = torch.zeros(8, 4, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    bad = [
        lambda: C.route(r, z.cpu()), lambda: C.route(r, z.half()), lambda: C.route(r, z[:, :32]), lambda: C.route(r, z.t()),
        lambda: C.route(r, z, bias=torch.zeros(63, device=DEV)), lambda: C.route(r, z, bias=torch.zeros(64)),
        lambda: C.route(r, z, ws=torch.zeros(256, dtype=torch.uint8, device=DEV)),
        lambda: C.route(r, z, ws=torch.zeros(1 << 20, dtype=torch.uint8)),
        lambda: C.route(r, z, ws=torch.zeros(1 << 20, device=DEV)),
        lambda: C.route(r, z, out=C.route(r, z[:4])), lambda: C.quantize_fp4(z.half()), lambda: C.quantize_fp4(z[:, :48]),
        lambda: C.quantize_fp4(z, 7), lambda: C.quantize_fp4(z, scale_exp=1 << 32),
        lambda: C.quantize_fp4(z, offsets=off, src_rows=pos[0], src_div=(1 << 32) + 1),
        lambda: C.quantize_fp4(z, src_rows=pos[0]), lambda: C.quantize_fp4(z.cpu()),
        lambda: C.quantize_fp4(z.expand(2, 8, 64)), lambda: C.quantize_fp4(z, offsets=off.long()),
        lambda: C.quantize_fp4(z, offsets=off, src_rows=pos[0].long()), lambda: C.quantize_fp4(z, out=C.quantize_fp4(z[:4])),
        lambda: C.dequantize_fp4(C.Fp4(0, torch.zeros(8, 32, device=DEV), torch.zeros(512, dtype=torch.uint8, device=DEV))),
        lambda: C.dequantize_fp4(C.Fp4(0, torch.zeros(8, 32, dtype=torch.uint8, device=DEV), torch.zeros(511, dtype=torch.uint8, device=DEV))),
        lambda: C.dequantize_fp4(C.quantize_fp4(z), out=torch.empty(8, 64, device=DEV)),
        lambda: C.moe_combine(y.float(), pos, w), lambda: C.moe_combine(y, pos.long(), w), lambda: C.moe_combine(y, pos, w[:4]),
        lambda: C.moe_combine(y, pos, w, x=torch.zeros(8, 32, device=DEV)), lambda: C.moe_combine(y[:, :60], pos, w),
        lambda: C.moe_combine(y, pos, w, shared=torch.zeros(8, 64, device=DEV)),
        lambda: C.moe_combine(torch.zeros(4, 12, dtype=torch.bfloat16, device=DEV), pos, w),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(C.CloverError):
            f()
            pytest.fail(f"call {i} was accepted")
