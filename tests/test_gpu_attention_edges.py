"""The attention operations at their edges, on the GPU: scores of any size, results that depend on nothing but what a
row sees."""
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


# ------------------------------------------- what a result may not depend on
#
# Compared bit for bit: out and lse.


def _equal(a, b, rows):
    for x, y in zip(a, b):
        assert torch.equal(x[rows].view(torch.uint8), y[rows].view(torch.uint8)), (x[rows] != y[rows]).float().mean()


def _cached_and_prompt(c, group):
    """Two calls of the same queries of one sequence: over its cache, and over 300 keys."""
    k, v = (torch.from_numpy(c.g.standard_normal((300, c.heads, c.dim))).bfloat16().to(DEV) for _ in range(2))
    off, ln, table = c.args()
    cache, koff = c.cache(), _ints([0, 300])
    return [lambda q: C.kv_attention(q, cache, off, ln, table, lse=True), lambda q: C.prompt_attention(q, k, v, off, koff, lse=True)]


@pytest.mark.parametrize("group,new", [(3, 40), (7, 40), (4, 50), (33, 5), (48, 5), (8, 1), (3, 4)])
@pytest.mark.parametrize("dim", [64, 128])
def test_rows_of_no_sequence_change_nothing(group, new, dim):
    c = Case([new], [300], 16, 2, dim, seed=group, extra_rows=64)
    q = c.q(2 * group)
    for call in _cached_and_prompt(c, group):
        first = call(q.to(DEV))
        for f in (0.0, 5.0, 100.0, float("nan")):
            x = q.clone()
            x[new:] *= f
            _equal(first, call(x.to(DEV)), slice(0, new))


@pytest.mark.parametrize("group,new", [(3, 40), (6, 40), (7, 40), (33, 5), (48, 5), (3, 4), (7, 2)])
@pytest.mark.parametrize("dim", [64, 128])
def test_calls_before_change_nothing(group, new, dim):
    """Groups that leave rows of a tile to what the kernel before had there."""
    c = Case([new], [300], 16, 2, dim, seed=group)
    q, other = c.q(2 * group).to(DEV), c.q(128)
    for call in _cached_and_prompt(c, group):
        got = []
        for f in (1e-3, 1.0, 5.0, 100.0):
            call((other * f).to(DEV))
            got.append(call(q))
        for x in got[1:]:
            _equal(got[0], x, slice(0, new))


@pytest.mark.parametrize("new,lens,heads,group,dim", [
    ([4] * 8, [12000 + i for i in range(8)], 2, 2, 64), ([5] * 8, [11000] * 8, 2, 3, 128),  # a few rows, a team per SM
    ([4] * 100, [1300 + i for i in range(100)], 2, 2, 64), ([2] * 100, [1300] * 100, 2, 6, 128),  # a piece per warp
    ([40], [900], 2, 8, 64), ([40], [1900], 1, 8, 128),  # tiles, cut
    ([40] * 40, [140] * 40, 4, 4, 64), ([40] * 40, [300] * 40, 4, 4, 128),  # whole
])
def test_cached_positions_behind_change_nothing(new, lens, heads, group, dim):
    """The last position's key, which only the last row of a sequence sees."""
    c = Case(new, lens, 16, heads, dim, seed=dim + len(new), written=False)
    c.pages[...] = c.g.integers(0, 256, c.pages.shape)
    for base in (0, 9 * dim):
        c.pages[..., base + 8 * dim:base + 9 * dim] = c.g.integers(28, 52, c.pages.shape[:3] + (dim,))
    q = c.q(heads * group).to(DEV)
    rows = torch.from_numpy(np.setdiff1d(np.arange(c.rows), c.off[1:] - 1)).to(DEV)
    first = C.kv_attention(q, c.cache(), *c.args(), lse=True)
    for byte in (0, 60, 70, 0x7F):
        for s, L in enumerate(lens):
            r = (L - 1) % 16
            c.pages[c.table[s, (L - 1) // 16], :, 0, 8 * dim + r * (dim // 16):8 * dim + (r + 1) * (dim // 16)] = byte
        _equal(first, C.kv_attention(q, c.cache(), *c.args(), lse=True), rows)


@pytest.mark.parametrize("new,lens,heads,group,dim", [([200], [200], 2, 4, 128), ([200], [200], 2, 8, 64), ([50], [2000], 1, 8, 64),
                                                      ([40] * 90, [140] * 90, 2, 8, 64), ([40] * 90, [300] * 90, 2, 8, 128)])
def test_prompt_positions_behind_change_nothing(new, lens, heads, group, dim):
    g = torch.Generator().manual_seed(dim)
    off, koff = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (new, lens))
    q = torch.randn((int(off[-1]), heads * group, dim), generator=g).bfloat16().to(DEV)
    k, v = (torch.randn((int(koff[-1]), heads, dim), generator=g).bfloat16().to(DEV) for _ in range(2))
    rows = torch.from_numpy(np.setdiff1d(np.arange(off[-1]), off[1:] - 1)).to(DEV)
    first = C.prompt_attention(q, k, v, _ints(off), _ints(koff), lse=True)
    last = torch.from_numpy(koff[1:] - 1).long().to(DEV)
    keys = k[last].clone()
    for f in (0.0, 10.0, 100.0, float("nan")):
        k[last] = keys * f
        _equal(first, C.prompt_attention(q, k, v, _ints(off), _ints(koff), lse=True), rows)


@pytest.mark.parametrize("group,dim", [(3, 64), (5, 128), (7, 64), (8, 128), (33, 64)])
def test_run_to_run(group, dim):
    """Every form of both operations, with calls of the others between two of a kind."""
    shapes = [([1], [1900]), ([1, 2, 1], [3000, 70, 900]), ([1] * 100, list(range(30, 330, 3))), ([40], [1500]), ([40] * 30, [90] * 30)]
    calls = []
    for i, (new, lens) in enumerate(shapes):
        c = Case(new, lens, 16, 4, dim, seed=i, written=False)
        c.pages[...] = c.g.integers(0, 0x38, c.pages.shape)  # (no NaN among the scales)
        q, cache, args = c.q(4 * group, 0.3).to(DEV), c.cache(), c.args()
        k = torch.from_numpy(c.g.standard_normal((sum(lens), 4, dim))).bfloat16().to(DEV)
        koff = _ints(np.concatenate([[0], np.cumsum(lens)]))
        calls.append(lambda q=q, cache=cache, args=args: C.kv_attention(q, cache, *args, lse=True))
        calls.append(lambda q=q, k=k, off=args[0], koff=koff: C.prompt_attention(q, k, k, off, koff, lse=True))
    first = [f() for f in calls]
    for i in range(4):
        for j in np.random.default_rng(i).permutation(len(calls)):
            _equal(first[j], calls[j](), slice(None))


# ---------------------------------- values that are not numbers, in large blocks


@pytest.mark.parametrize("block", [700, 333])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_odd_values_of_a_later_block(block, dim):
    """Tiles whose rows are of two blocks: the first rows must not get what the others see. Infinities of both signs and NaN,
    more than 32 positions apart and next to one another, at the ends of what is seen."""
    c = Case([1100], [1100], 16, 2, dim, seed=block, written=False)
    q = c.q(8)
    k, v = (torch.from_numpy(c.g.standard_normal((1100, 2, dim))).bfloat16() for _ in range(2))
    for p, d, x in ((block, 0, np.inf), (block + 40, 1, -np.inf), (block + 41, 1, -np.inf), (2 * block - 1, 33, np.nan),
                    (1099, dim - 1, np.inf), (1098, dim - 1, -np.inf), (block - 1, 20, np.inf)):
        if p < 1100:
            v[p, 1, d] = x
    off = _ints([0, 1100])
    out, lse = C.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), off, block=block, lse=True)
    want = R.prompt_attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), np.array([0, 1100]), np.array([0, 1100]),
                              block, dim ** -0.5)
    o, g = want[0], out.double().cpu().numpy()
    assert not np.isfinite(o).all()
    for same in (np.isnan, lambda x: x == np.inf, lambda x: x == -np.inf):
        assert np.array_equal(same(g), same(o))
    fine = np.isfinite(o)
    # the shorter tests' bound (scores below 64 here: d = 2^-13)
    assert (np.abs(g[fine] - o[fine]) <= 2.0 ** -8 * np.abs(o[fine]) + (2.0 ** -8 + 2.0 ** -13 + 2.0 ** -11) * want[2][fine]).all()


@pytest.mark.parametrize("block", [700, 333])
@pytest.mark.parametrize("dim", [64, 128])
def test_cached_odd_values_of_a_later_block(block, dim):
    c = Case([1100], [1100], 16, 2, dim, seed=block + 1, written=False)
    c.pages[...] = c.g.integers(0, 256, c.pages.shape)
    for base in (0, 9 * dim):
        c.pages[..., base + 8 * dim:base + 9 * dim] = c.g.integers(28, 52, c.pages.shape[:3] + (dim,))
    for p, d in ((block, 0), (block + 40, 1), (block + 41, 1), (2 * block - 1, 2), (1099, dim // 16 - 1), (block - 1, 3)):
        if p < 1100:
            c.pages[c.table[0, p // 16], 1, 0, 17 * dim + p % 16 * (dim // 16) + d] = 0x7F
    q = c.q(8)
    out, lse = C.kv_attention(q.to(DEV), c.cache(), *c.args(), block=block, lse=True)
    want = R.kv_attention(q.double().numpy(), c.pages, c.off, c.lens, c.table, block, dim ** -0.5)
    o, g = want[0], out.double().cpu().numpy()
    fine = ~np.isnan(o)
    assert not fine.all() and np.array_equal(np.isnan(g), ~fine)
    # (scores below 64: d = 2^-13)
    assert (np.abs(g - o)[fine] <= (2.0 ** -8 * np.abs(o) + (2.0 ** -12 + 2.0 ** -13 + 2.0 ** -11) * want[2] + 2.0 ** -36 * want[4])[fine]).all()


# ------------------------------------------------------------------- status


class _Words:
    def __init__(self, p):
        self.__cuda_array_interface__ = dict(shape=(64,), typestr="<i4", data=(p, False), version=2)


def test_status_without_a_workspace():
    """A set status word is reported once and cleared, whichever calls come between."""
    c = Case([1, 40], [70, 90], 16, 2, 64, seed=71)
    q, cache, args = c.q(8).to(DEV), c.cache(), c.args()
    k = torch.zeros((41, 2, 64), dtype=torch.bfloat16, device=DEV)
    p, n = C._attention_status()
    assert n == 256 and p % 256 == 0 and C._attention_status() == (p, n)
    want = C.kv_attention(q, cache, *args)
    C.prompt_attention(q, k, k, args[0])
    C.attention_status()
    word = torch.as_tensor(_Words(p), device=DEV)
    assert word.tolist() == [0] * 64
    word[0] = 1  # what a wait that ran out records
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(C.kv_attention(q, cache, *args), want)
    ws = C.workspace(C.kv_attention_workspace_bytes(cache, c.rows, 8, *args[2].shape))
    C.kv_attention(q, cache, *args, ws=ws)
    C.workspace_status(ws)
    C.prompt_attention(q, k, k, args[0], stream=side)
    with pytest.raises(C.CloverError) as e:
        C.attention_status(stream=side)
    assert e.value.code == C.ERR_DEVICE_TIMEOUT
    C.attention_status()
    assert word.tolist() == [0] * 64
