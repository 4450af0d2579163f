"""The grouped 4-bit product on the GPU against the fp64 oracle, and the
routed-expert operations run together. Every call goes through the C ABI.

Tolerances: products of e2m1 values and their scales are exact in fp32; the
tensor core's sum of K of them is given 2^-13 of the sum of the terms'
magnitudes (16 fp32 steps of 2^-24 for each of up to 128 instructions of 64
elements), the epilogue's SwiGLU a few fp32 steps on top, and the result's
rounding to bf16 2^-8 (half a step, relative to the value)."""
import numpy as np
import pytest
import torch

from block_diffusion_moe_gb300 import clover as C
from oracle import moe_ops as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMT = {"nv": C.FP4_NV, "mx": C.FP4_MX}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _values(q):
    """What an Fp4 stands for, fp64, by the dequantiser (checked bit for bit elsewhere)."""
    return C.dequantize_fp4(q).double().cpu()


def _operands(counts, N, K, fmt, swiglu, seed, extra_rows=0, scale_exp=0):
    """Quantised rows in groups of these sizes and a matrix (or gate and up) per group."""
    g = _gen(seed)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(off[-1]) + extra_rows
    x = torch.randn(n, K, generator=g) * torch.exp2(torch.randint(-3, 4, (n, 1), generator=g).float())
    mats, rows = (2 * len(counts), N // 2) if swiglu else (len(counts), N)
    w = torch.randn(mats, rows, K, generator=g) * 2.0 ** (scale_exp - 2)
    a = C.quantize_fp4(x.bfloat16().to(DEV), FMT[fmt], offsets=torch.from_numpy(off).to(DEV))
    b = C.quantize_fp4(w.bfloat16().to(DEV), FMT[fmt], scale_exp=scale_exp)
    return a, b, off


def _reference(a, b, off, swiglu, alpha=None):
    """(result, bound on its error) in fp64."""
    av, bv = _values(a)[: off[-1]], _values(b)
    G = len(off) - 1
    bv = bv.view(G, -1, a.cols)
    al = np.ones(G) if alpha is None else alpha
    ys, mags = [], []
    for i in range(G):
        r = slice(off[i], off[i + 1])
        ys.append(al[i] * (av[r] @ bv[i].T))
        mags.append(abs(al[i]) * (av[r].abs() @ bv[i].abs().T) * 2.0 ** -13)
    y, m = torch.cat(ys), torch.cat(mags)
    if swiglu:
        h = y.shape[1] // 2
        gate, up, mg, mu = y[:, :h], y[:, h:], m[:, :h], m[:, h:]
        s = gate / (1 + torch.exp(-gate))
        # |silu'| <= 1.1; exp and the quotient 2^-20 of the value
        y = s * up
        m = 1.1 * mg * up.abs() + s.abs() * mu + 1.1 * mg * mu + y.abs() * 2.0 ** -20
    return y, m + (y.abs() + m) * 2.0 ** -8 + 1e-37


def _check(a, b, off, swiglu=False, alpha=None, **kw):
    ws = C.workspace(C.fp4_product_workspace_bytes())
    out = torch.full((a.rows, b.rows), 7.0, dtype=torch.bfloat16, device=DEV)
    got = C.fp4_product(a, b, swiglu=swiglu, ws=ws, out=out, **kw)
    C.workspace_status(ws)
    y, tol = _reference(a, b, off, swiglu, alpha)
    err = (got[: off[-1]].double().cpu() - y).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), int((err > tol).sum()))
    assert got[off[-1]:].eq(7.0).all()
    return got


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("rows,N,K", [(1, 8, 64), (1, 256, 256), (128, 256, 256), (5, 100, 128), (130, 300, 320),
                                      (64, 1, 192), (200, 257, 2048), (300, 520, 1088), (1000, 1000, 448)])
def test_one_matrix(rows, N, K, fmt):
    a, b, off = _operands([rows], N, K, fmt, False, rows + N)
    _check(a, b, off)
    # without offsets: the same rows and layout as one matrix
    a.offsets = None
    _check(a, b, off)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("rows,N,K", [(1, 2, 64), (3, 256, 256), (128, 512, 512), (33, 128, 2048), (140, 420, 320), (257, 66, 128)])
def test_one_matrix_swiglu(rows, N, K, fmt):
    _check(*_operands([rows], N, K, fmt, True, rows + N), swiglu=True)


COUNTS = [[0, 1, 0, 0, 33, 128, 0, 129, 2, 0], [300, 0, 500, 1], [1] * 70, [0, 0, 5], [127, 1, 128, 255, 257], [0] * 3,
          [1, 0] * 256]


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts", COUNTS, ids=range(len(COUNTS)))
def test_groups(counts, swiglu, fmt):
    """Empty groups, groups that end inside a tile, more tiles than SMs, rows behind the last group."""
    a, b, off = _operands(counts, 384, 192, fmt, swiglu, len(counts), extra_rows=3)
    _check(a, b, off, swiglu=swiglu)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,N,K", [([256], 256, 256), ([512], 512, 64), ([300], 130, 320), ([1000, 0, 3], 520, 448),
                                        ([0, 513, 385, 1], 256, 192), ([700] * 40, 600, 320), ([129, 640], 96, 2048)])
def test_long_groups(counts, N, K, swiglu, fmt):
    """256 rows per group and more, several row tiles per group."""
    _check(*_operands(counts, N, K, fmt, swiglu, sum(counts), extra_rows=1), swiglu=swiglu)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("counts,N,K,swiglu", [([1024], 256, 8192, False), ([1100, 0, 2300], 520, 8192, False),
                                               ([1, 2400, 1000], 130, 8192, False), ([1150], 512, 4096, True),
                                               ([3000, 1, 129, 1000], 260, 4288, True), ([1025] * 3, 66, 4160, True)])
def test_pairs_of_ctas(counts, N, K, swiglu, fmt):
    """Long groups and a long K: tiles of 256 rows on two CTAs, with and without rows in the second half, and with a K
    that ends inside a stage."""
    _check(*_operands(counts, N, K, fmt, swiglu, sum(counts), extra_rows=2), swiglu=swiglu)


def test_scale_exponents_and_alpha():
    for swiglu in (False, True):
        a, b, off = _operands([40, 0, 90], 128, 256, "nv", swiglu, 3, scale_exp=-9)
        al = np.array([0.5, 3.0, -2.0])
        got = C.fp4_product(a, b, swiglu=swiglu, alpha=0.25, group_alpha=torch.tensor(al, dtype=torch.float32, device=DEV))
        y, tol = _reference(a, b, off, swiglu, al * 0.25)
        assert bool(((got.double().cpu() - y).abs() <= tol).all())


def test_long_sums():
    """K of 8,192: 128 instructions into one accumulator."""
    _check(*_operands([150], 260, 8192, "nv", False, 4))
    _check(*_operands([20, 140], 260, 8192, "mx", True, 4), swiglu=True)


def test_rows_do_not_depend_on_one_another():
    a, b, off = _operands([3, 200, 57], 300, 512, "nv", False, 5)
    whole = C.fp4_product(a, b)
    for g, r in ((0, slice(0, 3)), (1, slice(3, 203)), (2, slice(203, 260))):
        one = C.quantize_fp4(C.dequantize_fp4(a)[r].contiguous(), C.FP4_NV)
        m = C.quantize_fp4(C.dequantize_fp4(b)[g].contiguous(), C.FP4_NV)
        assert torch.equal(C.fp4_product(one, m), whole[r])
    for _ in range(5):
        assert torch.equal(C.fp4_product(a, b), whole)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_nan_stays_in_its_row_and_column(fmt):
    g = _gen(6)
    x, w = torch.randn(40, 128, generator=g), torch.randn(70, 128, generator=g)
    x[7, 50], w[33, 100] = float("nan"), float("inf")
    a, b = C.quantize_fp4(x.to(DEV), FMT[fmt]), C.quantize_fp4(w.to(DEV), FMT[fmt])
    y = C.fp4_product(a, b).cpu()
    bad = torch.zeros(40, 70, dtype=torch.bool)
    bad[7], bad[:, 33] = True, True
    assert torch.equal(y.isnan(), bad)


def test_offsets_out_of_range():
    a, b, off = _operands([10, 20], 64, 128, "nv", False, 7)
    want = C.fp4_product(a, b)
    a.offsets = torch.tensor([-5, 10, 1 << 30], dtype=torch.int32, device=DEV)
    assert torch.equal(C.fp4_product(a, b), want)
    a.offsets = torch.tensor([20, 10, 5], dtype=torch.int32, device=DEV)  # not ascending: no rows
    y = torch.full((30, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    assert C.fp4_product(a, b, out=y).eq(3.0).all()


def test_empty_and_refused():
    a, b, off = _operands([10, 20], 64, 128, "nv", False, 8)
    e = C.quantize_fp4(torch.zeros(0, 128, device=DEV), C.FP4_NV, offsets=torch.zeros(3, dtype=torch.int32, device=DEV))
    assert C.fp4_product(e, b).shape == (0, 64)
    m, _, _ = _operands([10, 20], 64, 128, "mx", False, 8)
    short, _, _ = _operands([10, 20], 64, 64, "nv", False, 8)
    one = C.Fp4(b.fmt, b.codes[0].contiguous(), b.scales)
    bad = [lambda: C.fp4_product(m, b), lambda: C.fp4_product(short, b), lambda: C.fp4_product(a, one),
           lambda: C.fp4_product(a, b, swiglu=True), lambda: C.fp4_product(b, b), lambda: C.fp4_product(a, a),
           lambda: C.fp4_product(a, b, out=torch.empty(30, 64, device=DEV)),
           lambda: C.fp4_product(a, b, group_alpha=torch.ones(3, device=DEV)),
           lambda: C.fp4_product(a, b, ws=torch.zeros(256, dtype=torch.uint8)),
           lambda: C.fp4_product(a, b, ws=torch.zeros(255, dtype=torch.uint8, device=DEV)),
           lambda: C.fp4_product(a, b, alpha=float("inf")), lambda: C.fp4_product(a, b, alpha=2.0 ** 128),
           lambda: C.fp4_product(a, C.Fp4(b.fmt, b.codes, b.scales[:-1])),
           lambda: C.fp4_product(a, C.Fp4(b.fmt, b.codes.cpu(), b.scales.cpu()))]
    for i, f in enumerate(bad):
        with pytest.raises(C.CloverError):
            f()
            pytest.fail(f"call {i} was accepted")


def test_results_past_2_31_elements():
    """Result rows that begin past 2^31 elements are those of the same rows alone."""
    rows, N, K = 270000, 8192, 64
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(rows, K, generator=g, device=DEV).bfloat16()
    b = C.quantize_fp4(torch.randn(N, K, generator=g, device=DEV).bfloat16(), C.FP4_MX)
    y = C.fp4_product(C.quantize_fp4(x, C.FP4_MX), b)
    for part in (slice(0, 200), slice(rows - 200, rows)):
        assert torch.equal(y[part], C.fp4_product(C.quantize_fp4(x[part].contiguous(), C.FP4_MX), b))


def test_many_row_tiles_and_column_tiles():
    """More tiles than SMs in both directions."""
    a, b, off = _operands([2000, 300, 1800], 1500, 256, "nv", False, 9)
    _check(a, b, off)


def _layer(x, xn, logits, bias, gate_up, down, K, fmt):
    """One routed-expert sublayer from the separate operations."""
    r = C.make_routing(logits.shape[1], K, score="sigmoid", n_groups=4, top_groups=2, group_rank=2, scale=1.5)
    sel = C.route(r, logits, bias=bias)
    a = C.quantize_fp4(xn, FMT[fmt], offsets=sel["offsets"], src_rows=sel["rows"], src_div=K)
    h = C.fp4_product(a, gate_up, swiglu=True)
    y = C.fp4_product(C.quantize_fp4(h, FMT[fmt], offsets=sel["offsets"]), down)
    return sel, h, C.moe_combine(y, sel["pos"], sel["w"], x=x)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M", [1, 32, 300])
def test_layer_together(M, fmt):
    """route -> quantize -> product with SwiGLU -> quantize -> product -> combine, against the oracle step by step (each
    step from the library's own input of that step, whose bits another test checks), and twice with the same bits."""
    E, K, H, F = 16, 4, 256, 128
    g = _gen(M)
    x = torch.randn(M, H, generator=g).to(DEV)
    xn = (x / x.square().mean(1, keepdim=True).sqrt()).bfloat16()
    logits = torch.randn(M, E, generator=g).to(DEV)
    if M > 4:
        logits[2] = -float("inf")
    bias = (0.1 * torch.randn(E, generator=g)).to(DEV)
    gate_up = C.quantize_fp4((0.06 * torch.randn(2 * E, F, H, generator=g)).bfloat16().to(DEV), FMT[fmt], scale_exp=-6)
    down = C.quantize_fp4((0.06 * torch.randn(E, H, F, generator=g)).bfloat16().to(DEV), FMT[fmt], scale_exp=-6)
    sel, h, out = _layer(x, xn, logits, bias, gate_up, down, K, fmt)
    ref = R.route(logits.cpu().numpy(), K, score="sigmoid", bias=bias.cpu().numpy(), n_groups=4, top_groups=2, group_rank=2, scale=1.5)
    assert np.array_equal(sel["idx"].cpu().numpy(), ref["idx"])
    n = int(ref["offsets"][-1])
    a = C.quantize_fp4(xn, FMT[fmt], offsets=sel["offsets"], src_rows=sel["rows"], src_div=K)
    rows = xn.float().cpu().numpy()[ref["rows"] // K]
    av = R.dequantize(*R.quantize(rows, fmt), fmt)
    assert np.array_equal(_values(a)[:n].numpy(), av)
    y, tol = _reference(a, gate_up, ref["offsets"], True)
    assert bool(((h[:n].double().cpu() - y).abs() <= tol).all())
    a2 = C.quantize_fp4(h, FMT[fmt], offsets=sel["offsets"])
    y, tol = _reference(a2, down, ref["offsets"], False)
    want = R.combine(y.numpy(), ref["pos"], ref["w"], x.cpu().numpy())
    off = R.combine(tol.numpy(), ref["pos"], np.abs(ref["w"]))
    mag = R.combine(y.abs().numpy(), ref["pos"], np.abs(ref["w"]), x.abs().cpu().numpy())
    assert np.all(np.abs(out.cpu().numpy() - want) <= off + mag * 2.0 ** -17)
    again = _layer(x, xn, logits, bias, gate_up, down, K, fmt)[2]
    assert torch.equal(again, out)
    # the quantisation itself: near the same layer without it
    exact = x.double().cpu().clone()
    w1 = C.dequantize_fp4(gate_up).double().cpu().view(E, 2 * F, H)
    w2 = C.dequantize_fp4(down).double().cpu()
    for t in range(M):
        for k in range(K):
            e = int(ref["idx"][t, k])
            if e >= 0:
                z = w1[e] @ xn[t].double().cpu()
                exact[t] += ref["w"][t, k] * (w2[e] @ (z[:F] / (1 + torch.exp(-z[:F])) * z[F:]))
    delta = exact - x.double().cpu()
    rel = (out.double().cpu() - exact).norm() / delta.norm().clamp(min=1e-30)
    assert rel < 0.3


def test_layer_captured():
    """The whole set in one graph, replayed on another stream with new inputs in place."""
    M, E, K, H, F = 64, 16, 4, 256, 128
    gate_up = C.quantize_fp4((0.06 * torch.randn(2 * E, F, H, generator=_gen(1))).bfloat16().to(DEV), C.FP4_NV, scale_exp=-6)
    down = C.quantize_fp4((0.06 * torch.randn(E, H, F, generator=_gen(2))).bfloat16().to(DEV), C.FP4_NV, scale_exp=-6)
    x = torch.randn(M, H, generator=_gen(3)).to(DEV)
    xn, logits, bias = x.bfloat16(), torch.randn(M, E, generator=_gen(4)).to(DEV), torch.zeros(E, device=DEV)
    args = (x, xn, logits, bias, gate_up, down, K, "nv")
    _layer(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = _layer(*args)[2]
    for seed in range(3):
        logits.copy_(torch.randn(M, E, generator=_gen(10 + seed)))
        xn.copy_(torch.randn(M, H, generator=_gen(20 + seed)))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert torch.equal(out, _layer(*args)[2])


def test_streams_at_once():
    """Products (single CTAs and pairs), routing and the framework's own layer kernel on three streams at the same time,
    each with its own workspace: the results of one after the other."""
    from block_diffusion_moe_gb300 import synth

    a1, b1, _ = _operands([40, 0, 300, 17], 700, 512, "nv", True, 31)
    a2, b2, _ = _operands([2100], 512, 8192, "nv", False, 32)  # long group, long K: CTA pairs
    d = synth.TINY
    layer, x = synth.make_layer(d, 33, 0, DEV), synth.make_x(d, 8, 34, DEV)
    z = torch.randn(3000, 256, generator=_gen(35)).to(DEV)
    r = C.make_routing(256, 8, score="sigmoid", n_groups=8, top_groups=4, group_rank=2)
    bias = (0.1 * torch.randn(256, generator=_gen(36))).to(DEV)
    ws = C.workspace(C.moe_workspace_bytes(d, 8))
    calls = [lambda: C.fp4_product(a1, b1, swiglu=True), lambda: C.fp4_product(a2, b2),
             lambda: C.route(r, z, bias=bias)["pos"], lambda: C.moe_block_step(d, layer, x, ws=ws, with_topk=False)[0]]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(10):
        for i, (f, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(f())
    torch.cuda.synchronize()
    C.workspace_status(ws)
    for i, w in enumerate(want):
        assert all(torch.equal(g, w) for g in got[i]), i
