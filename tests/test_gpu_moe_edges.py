"""The routed-expert operations at their edges. Every call goes through the C
ABI."""
import pytest
import torch

from block_diffusion_moe_gb300 import clover as C
from block_diffusion_moe_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


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
