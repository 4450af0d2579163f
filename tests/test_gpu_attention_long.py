"""Attention over so many positions that sums are flushed on the way (32,768 keys of one accumulator), on the GPU."""
import numpy as np
import pytest
import torch

from block_diffusion_moe_gb300 import clover as C
from tests.test_gpu_attention import DEV, _ints

pytestmark = pytest.mark.gpu

DIM = 64


def _pages(n, heads, seed, growing=False):
    """A cache of n positions, page j at position 64 j: keys whose scales grow along the positions, or anything; values of
    0.5 to 6 times a scale from 2^-4 to below 2, all positive."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pages = torch.randint(0, 256, (n // 64, heads, 4, 18 * DIM), generator=g, device=DEV, dtype=torch.uint8)
    k = torch.randint(24, 32, (n // 64, heads, 4, DIM), generator=g, device=DEV, dtype=torch.int32)
    if growing:
        k += (torch.arange(n // 64, device=DEV) * 16 // (n // 64))[:, None, None, None]
    pages[..., 8 * DIM:9 * DIM] = k.to(torch.uint8)
    codes = pages[..., 9 * DIM:17 * DIM]
    pages[..., 9 * DIM:17 * DIM] = (codes & 0x77).clamp(min=1) | 0x11
    pages[..., 17 * DIM:] = torch.randint(24, 64, (n // 64, heads, 4, DIM), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    return C.KvCache(pages)


def _values(cache, n, at=0):
    """Keys and values of positions at .. at + n - 1, bf16 (exact)."""
    table = torch.arange(at // 64, (at + n) // 64, device=DEV, dtype=torch.int32)[None]
    return C.kv_read(cache, _ints([0, n]), _ints([n]), table, n)


def _call(cache, seqs, new, q, n, **kw):
    table = torch.arange(n // 64, device=DEV, dtype=torch.int32)[None].expand(seqs, -1).contiguous()
    return C.kv_attention(q, cache, _ints(np.arange(seqs + 1) * new), _ints([n] * seqs), table, scale=DIM ** -0.5, lse=True, **kw)


# sequences, rows of each, heads, group, positions: as many as give every accumulator at least 40,000
FORMS = {
    "a piece per warp": (512, 1, 4, 4, 1 << 17), "a piece per warp, 16 rows": (300, 1, 4, 12, 1 << 17),
    "a team per SM": (47, 1, 4, 4, 1 << 20), "a team per SM, 16 rows": (37, 1, 4, 12, 1 << 20),
    "tiles, whole": (80, 4, 1, 64, 1 << 16), "tiles, cut": (19, 16, 1, 64, 1 << 17),
}
# (the last two for prompts, whose sequences have keys of their own: heads, rows, group, positions)
PROMPTS = {"whole": (1, 320, 64, 1 << 16), "cut": (1, 300, 64, 1 << 17)}


@pytest.mark.parametrize("form", ["a piece per warp", "a team per SM", "tiles, whole", "tiles, cut"])
def test_cached_means(form):
    """Equal scores: means of values of one sign. Sums may be off by 2^-13 of them. Results are rounded to bf16, by at most 2^-8
    of a value each; the mean of 256 (64 for one head) different ones, four standard deviations of a uniform error."""
    seqs, new, heads, group, n = {"a piece per warp": (512, 1, 4, 4, 1 << 21), "a team per SM": (47, 1, 4, 4, 1 << 24),
                                  "tiles, whole": (80, 4, 1, 64, 1 << 20), "tiles, cut": (19, 16, 1, 64, 1 << 21)}[form]
    cache = _pages(n, heads, 1)
    want = torch.zeros((heads, DIM), dtype=torch.float64, device=DEV)
    for at in range(0, n, 1 << 20):
        want += _values(cache, 1 << 20, at)[1].sum(0, dtype=torch.float64) / n
    q = torch.zeros((seqs * new, heads * group, DIM), dtype=torch.bfloat16, device=DEV)
    out, lse = _call(cache, seqs, new, q, n, block=0)
    err = (out.double().view(-1, heads, group, DIM) / want[:, None] - 1).mean().item()
    assert abs(err) <= 2.0 ** -13 + 4 * 2.0 ** -8 / (3 * heads * DIM) ** 0.5, err
    assert (lse.double() - np.log(n)).abs().max() <= 2.0 ** -17


@pytest.mark.parametrize("rows,n", [(320, 1 << 20), (300, 1 << 21)])  # whole, cut
def test_prompt_means(rows, n):
    g = torch.Generator(device=DEV).manual_seed(n)
    v = ((1 + torch.rand((n, 1, DIM), generator=g, device=DEV)) * (1 + torch.rand((1, 1, DIM), generator=g, device=DEV))).bfloat16()
    q = torch.zeros((rows, 64, DIM), dtype=torch.bfloat16, device=DEV)
    out, lse = C.prompt_attention(q, torch.zeros_like(v), v, _ints([0, rows]), _ints([0, n]), block=0, lse=True)
    err = (out.double() / v[:, 0].mean(0, dtype=torch.float64) - 1).mean().item()
    assert abs(err) <= 2.0 ** -13 + 4 * 2.0 ** -8 / (3 * DIM) ** 0.5, err
    assert (lse.double() - np.log(n)).abs().max() <= 2.0 ** -17


def _expected(q, k, v, lim):
    """One query over the first lim positions in fp64: out, lse, the sum of p |v|, the largest scale * sum |q k|, the sum of |v|."""
    k, v, q = k[:lim].double(), v[:lim].double(), q.double()
    z = k @ q * DIM ** -0.5
    p = torch.softmax(z, 0)
    return p @ v, torch.logsumexp(z, 0), p @ v.abs(), (k.abs() @ q.abs()).max() * DIM ** -0.5, v.abs().sum(0)


def _check(out, lse, want, half_step):
    """The bound of the shorter tests (test_gpu_attention), with the numerators' own half step."""
    o, z, mag, size, total = want
    d = 2.0 ** -19 * (1 + size)
    tol = 2.0 ** -8 * o.abs() + (half_step + 2.0 ** -13 + 4 * d) * mag + 2.0 ** -36 * total
    assert ((out.double() - o).abs() <= tol).all(), ((out.double() - o).abs() / tol).max()
    assert (lse.double() - z).abs() <= 2 * d + 2.0 ** -20 * z.abs() + 2.0 ** -13  # (the sum of weights: as other sums)


@pytest.mark.parametrize("form", FORMS)
def test_cached_results(form):
    """Maxima that grow along the positions; then a value that is not a number, which some rows see, or all."""
    seqs, new, heads, group, n = FORMS[form]
    cache = _pages(n, heads, 2, growing=True)
    k, v = _values(cache, n)
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn((seqs * new, heads * group, DIM), generator=g, device=DEV).bfloat16()
    out, lse = _call(cache, seqs, new, q, n, block=1)
    for row in (0, seqs * new // 2, seqs * new - 1):
        for h in (0, heads * group - 1):
            want = _expected(q[row, h], k[:, h // group], v[:, h // group], n - new + row % new + 1)
            _check(out[row, h], lse[row, h], want, 2.0 ** -12)
    # seen by the last row alone, in the first 16 elements
    cache.pages[-1, :, 3, 17 * DIM + 15 * (DIM // 16)] = 0x7F
    again, lse2 = _call(cache, seqs, new, q, n, block=1)
    last = torch.arange(seqs * new, device=DEV) % new == new - 1
    assert again[last][..., :16].isnan().all() and torch.equal(again[last][..., 16:], out[last][..., 16:])
    assert torch.equal(again[~last], out[~last]) and torch.equal(lse2, lse)
    # by all
    cache.pages[5, :, 1, 17 * DIM + 2] = 0x7F
    again, _ = _call(cache, seqs, new, q, n, block=1)
    assert again[..., 32:48].isnan().all() and torch.equal(again[..., 16:32], out[..., 16:32])


@pytest.mark.parametrize("form", PROMPTS)
def test_prompt_results(form):
    heads, rows, group, n = PROMPTS[form]
    g = torch.Generator(device=DEV).manual_seed(4)
    q = torch.randn((rows, heads * group, DIM), generator=g, device=DEV).bfloat16()
    k = (torch.randn((n, heads, DIM), generator=g, device=DEV) * torch.linspace(0.2, 2.0, n, device=DEV)[:, None, None]).bfloat16()
    v = torch.randn((n, heads, DIM), generator=g, device=DEV).bfloat16()
    call = lambda: C.prompt_attention(q, k, v, _ints([0, rows]), _ints([0, n]), block=1, lse=True)  # noqa: E731
    out, lse = call()
    for row in (0, rows // 2, rows - 1):
        for h in (0, heads * group - 1):
            want = _expected(q[row, h], k[:, h // group], v[:, h // group], n - rows + row + 1)
            _check(out[row, h], lse[row, h], want, 2.0 ** -8)
    v[-1, :, :16] = float("inf")
    again, lse2 = call()
    assert (again[-1, :, :16] == torch.inf).all() and torch.equal(again[-1, :, 16:], out[-1, :, 16:])
    assert torch.equal(again[:-1], out[:-1]) and torch.equal(lse2, lse)
