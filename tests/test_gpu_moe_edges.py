"""The routed-expert operations at their edges. Every call goes through the C
ABI."""
import numpy as np
import pytest
import torch

from block_diffusion_moe_gb300 import clover as C
from block_diffusion_moe_gb300 import synth
from oracle import moe_ops as R

from .test_gpu_fp4_product import _operands
from .test_gpu_moe_ops import _check_route

pytestmark = pytest.mark.gpu
DEV = "cuda"
LOWEST = torch.finfo(torch.float32).min


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# -------------------------------------------------------------------- streams


def _chain(x, logits, bias, gate_up, down, **kw):
    r = C.make_routing(logits.shape[1], 4, score="sigmoid", n_groups=4, top_groups=2, group_rank=2)
    sel = C.route(r, logits, bias=bias, **kw)
    a = C.quantize_fp4(x, C.FP4_NV, offsets=sel["offsets"], src_rows=sel["rows"], src_div=4, **kw)
    h = C.fp4_product(a, gate_up, swiglu=True, **kw)
    q = C.quantize_fp4(h, C.FP4_NV, offsets=sel["offsets"], **kw)
    y = C.fp4_product(q, down, **kw)
    return [sel[k] for k in ("idx", "w", "offsets", "rows", "pos")] + [C.dequantize_fp4(q, **kw), y,
                                                                     C.moe_combine(y, sel["pos"], sel["w"], **kw)]


def test_calls_on_a_stream_that_is_not_the_current_one():
    """stream= while the current stream is busy, fills and frees blocks of the calls' own sizes: the results of the same
    calls alone."""
    M, E, H, F = 3000, 16, 256, 128
    x, logits = torch.randn(M, H, generator=_gen(51)).bfloat16().to(DEV), torch.randn(M, E, generator=_gen(52)).to(DEV)
    bias = (0.1 * torch.randn(E, generator=_gen(53))).to(DEV)
    gate_up = C.quantize_fp4((0.06 * torch.randn(2 * E, F, H, generator=_gen(54))).bfloat16().to(DEV))
    down = C.quantize_fp4((0.06 * torch.randn(E, H, F, generator=_gen(55))).bfloat16().to(DEV))
    args = (x, logits, bias, gate_up, down)
    d = synth.TINY
    layer, xl = synth.make_layer(d, 33, 0, DEV), synth.make_x(d, 8, 34, DEV)
    want = _chain(*args)
    want_layer = C.moe_block_step(d, layer, xl, with_topk=False)[0]
    n_slots = int(want[2][-1])
    assert n_slots == M * 4
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    for _ in range(10):
        for _ in range(4):
            big = (big @ big).clamp(-1, 1)
        for n in (t.numel() * t.element_size() for t in want):
            torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV)
        got = _chain(*args, stream=side)
        got_layer = C.moe_block_step(d, layer, xl, with_topk=False, stream=side)[0]
        for n in (t.numel() * t.element_size() for t in want):
            torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV)
        side.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        assert torch.equal(got_layer, want_layer)
    torch.cuda.synchronize()


# -------------------------------------------------------------------- routing


@pytest.mark.parametrize("low", [-1e9, LOWEST])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masked_by_finite_biases(score, low):
    """Experts switched off (or forced) by a large finite bias: alone, a group of them, all but a few."""
    z = 1.5 * torch.randn(200, 256, generator=_gen(41))
    z[4, 30:] = -float("inf")
    b = 0.2 * torch.randn(256, generator=_gen(42))
    some, group, most, forced = b.clone(), b.clone(), b.clone(), b.clone()
    some[torch.randperm(256, generator=_gen(43))[:90]] = low
    group[32:64] = low
    most[5:250] = low
    forced[77], forced[100:110] = -low, low
    for bias in (some, group, most, forced):
        _check_route(z.to(DEV), dict(top_k=8, score=score), bias=bias.to(DEV))
        _check_route(z.to(DEV), dict(top_k=20, score=score), bias=bias.to(DEV))
        for rank in (1, 2):
            kw = dict(top_k=8, score=score, n_groups=8, top_groups=3, group_rank=rank)
            _check_route(z.to(DEV), kw, bias=bias.to(DEV))
            _check_route(z[:, :120].contiguous().to(DEV), dict(kw, n_groups=6), bias=bias[:120].contiguous().to(DEV))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [4, 3])
def test_route_group_ranks_outside_fp32(score, size):
    """Two biases whose sum leaves fp32's range either way: groups go by the sum itself, and a live group comes before
    one without an expert. (Groups of 4 lie on whole lanes, groups of 3 do not.)"""
    z = torch.randn(30, 6 * size, generator=_gen(44))
    z[3, :size] = -float("inf")
    z[5] = -float("inf")
    b = torch.empty(6 * size)
    for g, v in enumerate((-3e38, -2e38, -float("inf"), -2.5e38, -3.2e38, 0.1)):
        b[g * size:(g + 1) * size] = v
    for sign in (1.0, -1.0):
        for top in range(1, 6):
            for k in (2, 3 * size):
                _check_route(z.to(DEV), dict(top_k=k, score=score, n_groups=6, top_groups=top, group_rank=2),
                             bias=(sign * b).to(DEV))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 2, 5, 16, 20])
def test_route_true_ties_in_front_of_closer_keys(k, score):
    """Experts of the same logit and bias, and others so close above or below them that only fp64 tells: the tie must
    not hide those."""
    rng = np.random.default_rng(k)
    for E, values, bias in ((64, 2, 0.25), (64, 3, 1e4), (250, 3, 0.25), (250, 40, 1e4), (24, 2, 0.0)):
        z = (0.5 + 1e-6 * rng.integers(0, values, size=(60, E))).astype(np.float32)
        z[rng.random((60, E)) < 0.5] = -3.0
        z[3:6] = 0.5
        b = np.where(rng.random(E) < 0.1, bias + 0.125, bias).astype(np.float32)
        zt, bt = torch.from_numpy(z).to(DEV), torch.from_numpy(b).to(DEV)
        _check_route(zt, dict(top_k=min(k, E), score=score), bias=bt)
        if E != 64:
            _check_route(zt, dict(top_k=min(k, E), score=score, n_groups=2, top_groups=1, group_rank=1), bias=bt)


def _route_us(z, r, bias):
    out, ws = C.route(r, z, bias=bias), C.workspace(C.route_workspace_bytes(r, z.shape[0]))
    best = float("inf")
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        for _ in range(5):
            C.route(r, z, bias=bias, ws=ws, out=out)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 200)
    return best


def test_route_masks_cost_no_more_than_other_biases():
    """An expert masked by a large finite bias does not put every token's order in doubt."""
    z = 1.5 * torch.randn(32768, 256, generator=_gen(45)).to(DEV)
    b = 0.1 * torch.randn(256, generator=_gen(46))
    for kw in (dict(score="sigmoid", n_groups=8, top_groups=4, group_rank=2), dict(score="softmax")):
        r = C.make_routing(256, 8, **kw)
        plain = _route_us(z, r, b.to(DEV))
        for low in (-1e9, LOWEST):
            for at in (slice(0, 1), slice(32, 64), slice(0, 256, 3)):
                m = b.clone()
                m[at] = low
                assert _route_us(z, r, m.to(DEV)) < 2 * plain, (kw, low, at)


@pytest.mark.parametrize("M", [4864, 4865, 38912, 38913, 40960, 40961, 90000])
def test_route_of_many_tokens(M):
    """Where a CTA's tokens begin to grow (4,865), where the CTAs do (38,913), and more counts of an expert than a scan
    loads at once (40,961): the slots against a stable sort."""
    E, K = 24, 2
    z = torch.randn(M, E, generator=_gen(M)) + torch.linspace(-1, 1, E)
    z[torch.rand(M, generator=_gen(M + 1)) < 0.05] = -float("inf")
    out = C.route(C.make_routing(E, K), z.to(DEV))
    got = {k: v.cpu() for k, v in out.items()}
    top = torch.sort(z, dim=1, descending=True, stable=True)
    idx = torch.where(top.values[:, :K] > -float("inf"), top.indices[:, :K], -1)
    assert torch.equal(got["idx"].long(), idx)
    flat = idx.flatten()
    key = torch.where(flat >= 0, flat, E)
    order = torch.argsort(key, stable=True)
    n = int((flat >= 0).sum())
    pos = torch.full((M * K,), -1, dtype=torch.int64)
    pos[order[:n]] = torch.arange(n)
    assert torch.equal(got["rows"][:n].long(), order[:n])
    assert torch.equal(got["pos"].long().flatten(), pos)
    assert torch.equal(got["offsets"].long(), torch.searchsorted(key[order].contiguous(), torch.arange(E + 1)))
    w = torch.softmax(top.values[:, :K].double(), 1)
    # differences of logits up to 12, an exponential and a quotient: 60 u
    assert bool(((got["w"].double() - torch.where(idx >= 0, w, 0.0)).abs() <= 60 * 2.0 ** -24).all())


# --------------------------------------------------------------- quantisation


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_dequantize_every_scale(fmt):
    """Every code under every scale byte, times powers of two that lead out of the scale's own range and back."""
    n = 127 if fmt == "nv" else 256
    block = 16 if fmt == "nv" else 32
    codes = np.tile(np.arange(16, dtype=np.uint8), (n, 4))
    sb = np.repeat(np.arange(n, dtype=np.uint8)[:, None], 64 // block, 1)
    tiles = R.scale_tiles(-(-n // 128), 64 // block)
    for r in range(n):
        for b in range(64 // block):
            tiles[R.scale_place(r, b)] = sb[r, b]
    q = C.Fp4(C.FP4_NV if fmt == "nv" else C.FP4_MX, torch.from_numpy(R.pack_codes(codes)).to(DEV),
              torch.from_numpy(tiles.reshape(-1)).to(DEV))
    for exp in (0, -1, -3, -64, 5, 64):
        q.scale_exp = exp
        want = torch.from_numpy(R.dequantize(codes, sb, fmt, exp)).bfloat16()
        got = C.dequantize_fp4(q).cpu()
        ok = (got == want) | (got.isnan() & want.isnan())
        assert bool(ok.all()), (exp, [int(r) for r in torch.nonzero(~ok.all(1)).flatten()][:5])


def test_refused_quantisation_leaves_out_as_it_was():
    """A refused call does not give `out` the exponent and offsets that its codes were not made for."""
    x = torch.randn(40, 72, generator=_gen(57)).to(DEV)
    off = torch.tensor([0, 30, 40], dtype=torch.int32, device=DEV)
    q = C.quantize_fp4(x[:, :64].contiguous(), scale_exp=-2, offsets=off)
    want = C.dequantize_fp4(q)
    with pytest.raises(C.CloverError):
        C.quantize_fp4(x[:, 1:65], scale_exp=5, offsets=torch.zeros(2, dtype=torch.int32, device=DEV), out=q)  # rows not aligned
    assert q.scale_exp == -2 and q.offsets is off and q.groups == 2
    assert torch.equal(C.dequantize_fp4(q), want)
    got = C.quantize_fp4(x[:, :64], scale_exp=5, offsets=off, out=q)
    assert got is q and q.scale_exp == 5
    assert torch.equal(C.dequantize_fp4(q), C.dequantize_fp4(C.quantize_fp4(x[:, :64], scale_exp=5)))


# -------------------------------------------------------------------- product


class _Words:
    def __init__(self, p):
        self.__cuda_array_interface__ = dict(shape=(64,), typestr="<i4", data=(p, False), version=2)


def test_product_without_workspace_keeps_its_status():
    """The status of a product without ws can be read afterwards: a set word is reported once and cleared, and a product
    uses that word (as every product does, on any stream) and leaves it alone."""
    a = C.quantize_fp4(torch.randn(70, 64, generator=_gen(61)).to(DEV))
    p, n = C._shared_workspace()
    assert n == C.fp4_product_workspace_bytes() and p % 256 == 0 and C._shared_workspace() == (p, n)
    want = C.fp4_product(a, a)
    C.fp4_product_status()
    word = torch.as_tensor(_Words(p), device=DEV)
    assert word.tolist() == [0] * 64
    word[0] = 1  # what a wait that ran out records
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(C.fp4_product(a, a), want)
    C.fp4_product(a, a, stream=side)
    with pytest.raises(C.CloverError) as e:
        C.fp4_product_status(stream=side)
    assert e.value.code == C.ERR_DEVICE_TIMEOUT
    C.fp4_product_status()
    assert word.tolist() == [0] * 64


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_swiglu_of_gates_far_below_zero(fmt):
    """silu falls to 0 for gates far below zero, whatever they are multiplied with. Rows and matrices have one element
    each, so that the products are exact."""
    up = 1.5 * 2.0 ** 9
    x = torch.zeros(40, 64)
    x[:, 0] = torch.tensor([1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -1.0, -6.0]).repeat(5) * torch.exp2(torch.arange(5.0)).repeat_interleave(8)
    w = torch.zeros(2, 8, 64)
    w[0, :, 0] = -4.0  # gate
    w[1, :, 0] = up
    a, b = C.quantize_fp4(x.to(DEV), C.FP4_NV if fmt == "nv" else C.FP4_MX), C.quantize_fp4(w.to(DEV), C.FP4_NV if fmt == "nv" else C.FP4_MX)
    av, wv = R.dequantize(*R.quantize(x.numpy(), fmt), fmt)[:, 0], R.dequantize(*R.quantize(w.view(16, 64).numpy(), fmt), fmt)[:, 0]
    for alpha in (1.0, 0.9375, 0.92, 1e3, 1e10, 1e20, 1e30):
        z = float(np.float32(alpha)) * np.outer(av, wv)
        gate, u = z[:, :8], z[:, 8:]
        with np.errstate(over="ignore", under="ignore"):
            y = gate / (1.0 + np.exp(-gate)) * u
            # the gate's rounding moves silu(g) by |g| u of its slope, the exponential's argument by 2 |g| u more, which
            # changes it in proportion (below 88; further down it is 0 but for denormals); a few steps of the rest
            rel = 2.0 ** -8 + (np.minimum(np.abs(gate), 128.0) * 4 + 16) * 2.0 ** -24
        got = C.fp4_product(a, b, swiglu=True, alpha=alpha).double().cpu().numpy()
        ordinary = np.abs(y) < 3e38
        assert np.all(np.abs(got - y)[ordinary] <= (rel * np.abs(y) + 2.0 ** -126 * np.maximum(np.abs(u), 1.0))[ordinary]), alpha
        assert np.all(np.abs(got[~ordinary]) >= 3e38)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("counts,N,K,swiglu", [([2100, 0, 2500], 2300, 8192, False), ([2100, 1, 2500], 2600, 4160, True),
                                               ([1500, 3100], 5000, 8192, False)])
def test_pairs_of_ctas_take_several_tiles(counts, N, K, swiglu, fmt):
    """More tiles than twice the pairs of CTAs: every pair uses both accumulators, and some the first again."""
    a, b, off = _operands(counts, N, K, fmt, swiglu, sum(counts), extra_rows=2)
    step = 128 if swiglu else 256
    width = N // 2 if swiglu else N
    tiles = sum(-(-c // 256) for c in counts) * -(-width // step)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert tiles > 2 * (sms // 2)
    ws = C.workspace(C.fp4_product_workspace_bytes())
    out = torch.full((a.rows, width), 7.0, dtype=torch.bfloat16, device=DEV)
    C.fp4_product(a, b, swiglu=swiglu, ws=ws, out=out)
    C.workspace_status(ws)
    assert out[off[-1]:].eq(7.0).all()
    av, bv = C.dequantize_fp4(a).double(), C.dequantize_fp4(b).double().view(len(counts), -1, K)
    for g in range(len(counts)):
        r = slice(off[g], off[g + 1])
        y, m = av[r] @ bv[g].T, av[r].abs() @ bv[g].abs().T * 2.0 ** -13
        if swiglu:
            gate, up, mg, mu = y[:, :width], y[:, width:], m[:, :width], m[:, width:]
            s = gate / (1 + torch.exp(-gate))
            y = s * up  # |silu'| <= 1.1; exp and the quotient 2^-20 of the value
            m = 1.1 * mg * up.abs() + s.abs() * mu + 1.1 * mg * mu + y.abs() * 2.0 ** -20
        tol = m + (y.abs() + m) * 2.0 ** -8 + 1e-37
        err = (out[r].double() - y).abs()
        assert bool((err <= tol).all()), (g, float((err / tol).max()), int((err > tol).sum()))
