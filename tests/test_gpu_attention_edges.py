"""The attention operations at their edges, on the GPU: scores of any size."""
import numpy as np
import pytest
import torch

from block_diffusion_moe_gb300 import clover as C
from oracle import attention as R
from tests.test_gpu_attention import DEV, Case, _ints

pytestmark = pytest.mark.gpu


def _near(got, lse, want, cached):
    """Results whose scores are exact in fp32, against the oracle's. The exponent c (S - max) is then off by the roundings of
    c and of the product, 2^-22 of itself, which changes p by less than 2^-22; each move of the maximum and each join adds
    as much, fewer than 32 of them: 2^-17 of p in all, and as much again through the sum of p. Numerators are rounded by
    2^-12 (cached, fp16) or 2^-8 (bf16) of each, or by 2^-36 of the largest; sums take 2^-13 of the sum of p |v|, the
    result's rounding to bf16 2^-8 of it. lse: 2^-17 for the sum of p, three roundings of 2^-24 for c max, two more for
    what follows."""
    out, z, mag, _, total = want
    g = got.double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(out) + ((2.0 ** -12 if cached else 2.0 ** -8) + 2.0 ** -13 + 2.0 ** -16) * mag \
        + 2.0 ** -130 + cached * 2.0 ** -36 * total
    bad = ~(np.abs(g - out) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:3], g[bad][:5], out[bad][:5], tol[bad][:5])
    g = lse.double().cpu().numpy()
    bad = ~(np.abs(g - z) <= 2.0 ** -17 + 2.0 ** -21 * np.abs(z))
    assert not bad.any(), (np.argwhere(bad)[:3], g[bad][:5], z[bad][:5])


# Scores scale * (+-6 * 2^18 +- w), w a multiple of 1/4 up to 6: exact in fp32 (21 bits), and 2^20 to 2^121 large. With the
# smaller scales several positions have a share, with the larger ones those that are largest have all.
SCALES = [2.0 ** e for e in (0, 4, 8, 14, 40, 100)]


def _large_queries(g, shape):
    q = torch.zeros(shape)
    q[..., 0] = 2.0 ** 18 * torch.from_numpy(g.choice([-1.0, 1.0], shape[:2]))
    q[..., 16] = torch.from_numpy(g.choice([-1.0, 1.0, 0.5], shape[:2]))
    return q.bfloat16()


@pytest.mark.parametrize("new,lens,heads,group,dim", [
    ([1], [1500], 2, 8, 128), ([1], [700], 2, 12, 64),                   # a few rows, a team per SM
    ([1] * 100, list(range(20, 120)), 2, 4, 64), ([1] * 100, list(range(20, 120)), 2, 12, 128),  # a piece per warp
    ([40], [1500], 2, 8, 64), ([34], [300], 1, 16, 128),                 # tiles, cut
    ([40] * 12, list(range(50, 62)), 8, 8, 64),                          # whole
])
def test_cached_scores_of_any_size(new, lens, heads, group, dim):
    c = Case(new, lens, 32, heads, dim, seed=len(new) + dim)
    for s, L in enumerate(lens):
        p = np.arange(L)
        pg, six, r = c.table[s, p // 32], p % 32 // 16, p % 16
        for i in range(dim // 2):
            c.pages[pg, :, six, r * (dim // 2) + i] = 0
        c.pages[pg, :, six, r * (dim // 2)] = 7                                      # element 0: 6
        c.pages[pg, :, six, r * (dim // 2) + 8] = c.g.integers(0, 16, (L, heads))    # element 16: any
        for i in range(dim // 16):
            c.pages[pg, :, six, 8 * dim + r * (dim // 16) + i] = 0x38                # scales of 1
    q = _large_queries(c.g, (c.rows, heads * group, dim))
    for scale in SCALES:
        want = R.kv_attention(q.double().numpy(), c.pages, c.off, c.lens, c.table, 1, scale)
        _near(*C.kv_attention(q.to(DEV), c.cache(), *c.args(), scale=scale, lse=True), want, True)


@pytest.mark.parametrize("new,lens,heads,group,dim", [
    ([200], [200], 2, 4, 128), ([200], [200], 2, 8, 64), ([1, 7, 150], [900, 70, 1000], 1, 8, 64),  # cut
    ([90] * 8, [90] * 8, 8, 8, 64), ([90] * 8, [90] * 8, 8, 8, 128),                                # whole
])
def test_prompt_scores_of_any_size(new, lens, heads, group, dim):
    g = np.random.default_rng(dim + heads)
    off, koff = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (new, lens))
    q = _large_queries(g, (int(off[-1]), heads * group, dim))
    k = torch.zeros(int(koff[-1]), heads, dim)
    k[..., 0] = 6
    k[..., 16] = torch.from_numpy(g.choice([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -1.0, -3.0, -6.0], k.shape[:2]))
    k, v = k.bfloat16(), torch.from_numpy(g.standard_normal(k.shape)).bfloat16()
    for scale in SCALES:
        want = R.prompt_attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), off, koff, 1, scale)
        _near(*C.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), _ints(off), _ints(koff), scale=scale, lse=True), want, False)
