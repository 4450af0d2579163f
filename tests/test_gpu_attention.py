"""The attention operations on the GPU against the fp64 oracle. Every call goes
through the C ABI.

Tolerances. Codes, scales and what is read back: equal, bit for bit. Attention:
products of 16-bit values are exact in fp32; a score's sum of up to 128 of them,
its scaling and the exponent are given d = 2^-19 (1 + the largest scale * sum
|q k| of a visible position) in absolute terms, which changes every p by a factor
within 1 +- 2 d and the softmax by as much again; numerators are rounded to 16
bits (bf16 at worst: half a step, 2^-8 of each); sums over positions and the
join of parts in fp32 take 2^-13 of the sum of p |v|; the result's rounding to bf16
is 2^-8 of the value:
  |out - exact| <= 2^-8 |exact| + (2^-8 + 2^-13 + 4 d) sum p |v|  (+ bf16's smallest steps)
  |lse - exact| <= 2 d + 2^-20 |exact|
Over the cache numerators are fp16, whose steps do not shrink below 2^-24. They are
lifted by 2^11 over the row's running maximum, which one numerator at least equals
(the sum of weights is 2^11 or more), so half such a step is 2^-36 of that sum:
  + 2^-36 sum |v| over the positions a query sees.
"""
import numpy as np
import pytest
import torch

from block_diffusion_moe_gb300 import clover as C
from oracle import attention as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _close(got, want, rows, lse=None, cached=False):
    """Checks the first `rows` rows of a result [n][Hq][D] (and lse) against the oracle's."""
    out, z, mag, size, total = (x[:rows] for x in want)
    g = got[:rows].float().cpu().numpy().astype(np.float64)
    d = 2.0 ** -19 * (1 + size)[..., None]
    with np.errstate(invalid="ignore"):
        tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -13 + 4 * d) * mag + 2.0 ** -130 + cached * 2.0 ** -36 * total
        err = np.abs(g - out)
    fine = np.isfinite(out)
    bad = fine & ~(err <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], g[bad][:5], out[bad][:5], tol[bad][:5])
    assert np.array_equal(g[~fine], out[~fine], equal_nan=True), np.argwhere(~fine)[:5]
    if lse is not None:
        s = lse[:rows].cpu().numpy().astype(np.float64)
        none, some = z == -np.inf, np.isfinite(z)
        assert (s[none] == -np.inf).all() and (g[none] == 0).all()
        assert (np.abs(s[some] - z[some]) <= 2 * d[..., 0][some] + 2.0 ** -20 * np.abs(z[some])).all()
        assert np.isnan(s[~none & ~some]).all()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Case:
    """Sequences with pages in a pool of random bytes (NaN scales among them): nothing but their own positions may matter."""

    def __init__(self, new, lens, page=32, kv_heads=2, dim=128, seed=0, extra_rows=0, k_exp=0, v_exp=0, written=True,
                 spare=2, max_pages=None):
        g = np.random.default_rng(seed)
        self.new, self.lens, self.dim, self.heads = new, lens, dim, kv_heads
        used = [-(-max(L, 0) // page) for L in lens]
        n = sum(used) + spare
        self.off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows = int(self.off[-1]) + extra_rows
        width = max(used + [1]) if max_pages is None else max_pages
        ids = g.permutation(n)
        self.table = np.full((len(new), width), -1, dtype=np.int32)
        at = 0
        for s, u in enumerate(used):
            self.table[s, :u] = ids[at:at + u]
            at += u
        self.pages = g.integers(0, 256, (n, kv_heads, page // 16, 18 * dim)).astype(np.uint8)
        self.g, self.k_exp, self.v_exp = g, k_exp, v_exp
        if written:  # plausible scales where positions are
            for s, L in enumerate(lens):
                for p in range(max(L, 0)):
                    pg, six, r = self.table[s, p // page], p % page // 16, p % 16
                    for base in (0, 9 * dim):
                        sc = self.pages[pg, :, six, base + 8 * dim + r * (dim // 16):base + 8 * dim + (r + 1) * (dim // 16)]
                        sc[:] = g.integers(28, 52, sc.shape)

    def cache(self):
        return C.KvCache(torch.from_numpy(self.pages).to(DEV), self.k_exp, self.v_exp)

    def args(self):
        return _ints(self.off), _ints(self.lens), _ints(self.table)

    def q(self, q_heads, std=1.0):
        return torch.from_numpy(std * self.g.standard_normal((self.rows, q_heads, self.dim))).bfloat16()

    def check(self, q_heads, block, scale=None, std=1.0):
        q = self.q(q_heads, std)
        sc = self.dim ** -0.5 if scale is None else scale
        want = R.kv_attention(q.double().numpy(), self.pages, self.off, self.lens, self.table, block, sc, self.k_exp, self.v_exp)
        mark = torch.full((self.rows, q_heads, self.dim), 7.0, dtype=torch.bfloat16, device=DEV)
        out, lse = C.kv_attention(q.to(DEV), self.cache(), *self.args(), block=block, scale=scale, lse=True, out=mark.clone())
        last = int(self.off[-1])
        _close(out, want, last, lse, cached=True)
        assert torch.equal(out[last:], mark[last:])
        return out, lse


# -------------------------------------------------------- writing and reading


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,lens,page,heads,dim", [
    ([1], [1], 16, 1, 64), ([1], [1000], 32, 2, 128), ([5, 0, 17, 1], [5, 3, 100, 64], 16, 3, 64),
    ([40, 33], [40, 95], 48, 2, 128), ([130], [130], 128, 1, 128), ([3, 2], [2, 0], 16, 2, 64),
])
def test_write_is_exact(dtype, new, lens, page, heads, dim):
    c = Case(new, lens, page, heads, dim, seed=page + dim, extra_rows=3, written=False, k_exp=1, v_exp=-2)
    shape = (c.rows, heads, dim)
    k, v = (torch.from_numpy(c.g.standard_normal(shape) * np.exp2(c.g.integers(-6, 7, shape[:2] + (1,)))).to(dtype)
            for _ in range(2))
    k[0, 0, :3] = torch.tensor([6.0, -3.0, 0.5]).to(dtype)
    cache = c.cache()
    C.kv_write(cache, k.to(DEV), v.to(DEV), *c.args())
    want = R.write(c.pages, k.double().numpy(), v.double().numpy(), c.off, c.lens, c.table, 1, -2)
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    mark = torch.full(shape, 7.0, dtype=torch.bfloat16, device=DEV)
    out = C.kv_read(cache, *c.args(), c.rows, out=(mark.clone(), mark.clone()))
    for s, r, i, n in R.rows_of(c.off, c.rows):
        p = lens[s] - n + i
        if p < 0:
            assert not out[0][r].any() and not out[1][r].any()
            continue
        kk, vv, _ = R.positions(want, c.table[s], p + 1, 1, -2)
        for got, ref in zip(out, (kk, vv)):
            assert np.array_equal(got[r].double().cpu().numpy(), ref[p])
    for got in out:
        assert torch.equal(got[c.off[-1]:], mark[c.off[-1]:])


def test_write_strided_rows_and_ends_of_the_format():
    """Keys and values side by side in one projection; blocks of zeros, of infinities and NaN, past the largest scale."""
    c = Case([37], [50], 16, 2, 64, seed=3, written=False)
    qkv = torch.from_numpy(c.g.standard_normal((37, 8, 64)) * 3).bfloat16()
    qkv[3, 4:] = 0
    qkv[4, 4, 5] = float("inf")
    qkv[5, 6, 17] = float("nan")
    qkv[6, 4:] *= 1e30
    qkv[7, 4:] *= 1e-30
    dev = qkv.to(DEV)
    cache = c.cache()
    C.kv_write(cache, dev[:, 4:6], dev[:, 6:8], *c.args())
    want = R.write(c.pages, qkv[:, 4:6].double().numpy(), qkv[:, 6:8].double().numpy(), c.off, c.lens, c.table)
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    # head-major rows, 16-byte but not 32-byte aligned
    raw = torch.empty(2 * 37 * 72 + 8, dtype=torch.bfloat16, device=DEV)
    hm = raw[8:].view(2, 37, 72)[:, :, :64].permute(1, 0, 2)
    hm.copy_(dev[:, 4:6])
    cache2 = c.cache()
    C.kv_write(cache2, hm, dev[:, 6:8], *c.args())
    assert torch.equal(cache2.pages, cache.pages)


def test_pages_that_are_not_there():
    c = Case([60], [60], 16, 2, 64, seed=4, written=False)
    c.table[0, 1], c.table[0, 2] = -1, c.pages.shape[0]
    k = torch.from_numpy(c.g.standard_normal((60, 2, 64))).bfloat16()
    cache = c.cache()
    C.kv_write(cache, k.to(DEV), k.to(DEV), *c.args())
    want = R.write(c.pages, k.double().numpy(), k.double().numpy(), c.off, c.lens, c.table)
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    out = C.kv_read(cache, *c.args(), 60)
    assert not out[0][16:48].any() and out[0][:16].any() and out[0][48:].any()


def test_write_through_a_large_pool():
    """Pages past 2^32 bytes."""
    n = (5 << 30) // C.kv_page_bytes(256, 2, 128)
    cache = C.KvCache.empty(n, 256, 2, 128)
    table = _ints([[n - 1, 0, n - 2]])
    k = torch.randn(700, 2, 128, device=DEV).bfloat16()
    off, lens = _ints([0, 700]), _ints([700])
    C.kv_write(cache, k, 2 * k, off, lens, table)
    kk, vv = C.kv_read(cache, off, lens, table, 700)
    assert torch.equal(vv, 2 * kk) and float((kk - k).float().norm() / k.float().norm()) < 0.15
    small = C.KvCache.empty(3, 256, 2, 128)
    t2 = _ints([[1, 2, 0]])
    C.kv_write(small, k, 2 * k, off, lens, t2)
    q = torch.randn(33, 16, 128, device=DEV).bfloat16()
    o2 = _ints([0, 33])
    assert torch.equal(C.kv_attention(q, cache, o2, lens, table), C.kv_attention(q, small, o2, lens, t2))
    del cache
    torch.cuda.empty_cache()


# ------------------------------------------------------ attention over a cache


@pytest.mark.parametrize("block", [0, 1, 32])
@pytest.mark.parametrize("new,lens,page,heads,group,dim", [
    ([1], [1], 16, 1, 1, 64), ([1], [17], 16, 2, 8, 128), ([1], [1021], 32, 2, 8, 128), ([1, 1, 1], [5, 300, 64], 64, 8, 4, 128),
    ([1, 1], [129, 1], 48, 1, 16, 64), ([2, 5, 1], [40, 5, 200], 16, 2, 5, 128), ([32], [500], 64, 2, 8, 128),
    ([32, 7, 0, 32], [64, 33, 10, 300], 16, 4, 8, 64), ([300], [300], 32, 1, 3, 128), ([70, 1], [200, 1500], 128, 1, 64, 64),
    ([33], [700], 16, 3, 7, 128), ([1], [333], 16, 1, 33, 128), ([150], [400], 16, 1, 1, 64),
])
def test_cached_attention(new, lens, page, heads, group, dim, block):
    for extra in (0, 2):  # (rows of no sequence can change which kernel takes the call)
        c = Case(new, lens, page, heads, dim, seed=sum(lens) + group, extra_rows=extra, k_exp=2, v_exp=-1)
        c.check(heads * group, block)


@pytest.mark.parametrize("new,group", [(1, 4), (9, 8)])
def test_cached_rows_that_see_nothing(new, group):
    """Lengths of zero, below the rows, below zero, past the table; sequences without rows."""
    c = Case([new, new, new, new, 0], [0, new // 2, 70, 40, 12], 16, 2, 64, seed=5)
    c.lens = [0, new // 2, 1 << 30, -5, 12]
    c.table[2, :] = c.g.integers(0, c.pages.shape[0], c.table.shape[1])
    c.pages[..., 8 * 64:9 * 64] &= 0x37
    c.pages[..., 17 * 64:] &= 0x37
    for block in (0, 1, 8):
        c.check(2 * group, block)


@pytest.mark.parametrize("group", [2, 16])
def test_cached_pages_that_are_not_there(group):
    c = Case([3, 20, 1], [100, 260, 90], 16, 2, 128, seed=6)
    c.table[0, 2], c.table[1, 5:9], c.table[1, 0], c.table[2, :] = -1, c.pages.shape[0] + 5, -7, -1
    for block in (0, 1):
        c.check(2 * group, block)


@pytest.mark.parametrize("new,group", [(1, 8), (6, 2), (32, 8)])
def test_cached_nan_where_it_is_seen_and_not_elsewhere(new, group):
    """A NaN scale of a value or a key reaches exactly the queries that see its position."""
    for value, at in ((1, 60), (0, 61), (1, 63), (0, 40)):
        c = Case([new, 1], [64, 50], 16, 1, 64, seed=at)
        base = (17 if value else 8) * 64 + at % 16 * 4
        c.pages[c.table[0, at // 16], 0, 0, base + 1] = 0x7F
        c.check(group, 1)
        c.check(group, 4)


@pytest.mark.parametrize("std,scale", [(30.0, None), (1.0, 40.0), (1e-3, 1e-3), (1e30, 1e-30), (1e-30, 1e29)])
def test_cached_extreme_scores(std, scale):
    for new, group in ((1, 8), (16, 8)):
        Case([new], [300], 32, 1, 128, seed=7).check(group, 1, scale, std)


def test_cached_peaks_in_any_order():
    """The largest score first, last and growing all the way."""
    for order in ("first", "last", "growing"):
        for new, group in ((1, 4), (32, 4)):
            c = Case([new], [600], 32, 1, 64, seed=8)
            for p in range(600):
                sc = c.pages[c.table[0, p // 32], 0, p % 32 // 16, 512 + p % 16 * 4:512 + p % 16 * 4 + 4]
                sc[:] = {"first": 90 if p == 0 else 30, "last": 90 if p == 599 else 30, "growing": 20 + p // 10}[order]
            c.check(group, 0, 1.0)


def _decoded(cache, table_row, length):
    """Keys and values of one sequence in fp64 on the GPU, by the reader (checked bit for bit above)."""
    off = _ints([0, length])
    k, v = C.kv_read(cache, off, _ints([length]), table_row[None].contiguous(), length)
    return k.double(), v.double()


@pytest.mark.parametrize("new,length,heads,group", [(1, 131072, 2, 8), (32, 131072, 2, 8), (1, 70001, 1, 1), (5, 33333, 4, 7)])
def test_cached_long_context(new, length, heads, group):
    g = torch.Generator(device=DEV).manual_seed(length)
    pages = -(-length // 64)
    cache = C.KvCache.empty(pages, 64, heads, 128)
    table = torch.randperm(pages, generator=g, device=DEV).int()[None]
    k, v = (torch.randn((length, heads, 128), generator=g, device=DEV).bfloat16() for _ in range(2))
    C.kv_write(cache, k, v, _ints([0, length]), _ints([length]), table)
    k, v = _decoded(cache, table[0], length)
    q = torch.randn((new, heads * group, 128), generator=g, device=DEV).bfloat16()
    out, lse = C.kv_attention(q, cache, _ints([0, new]), _ints([length]), table, lse=True)
    for h in range(heads * group):
        z = q[:, h].double() @ k[:, h // group].T * 128 ** -0.5
        z.masked_fill_(torch.arange(length, device=DEV) > torch.arange(length - new, length, device=DEV)[:, None], -torch.inf)
        p = torch.softmax(z, 1)
        want, mag = p @ v[:, h // group], p @ v[:, h // group].abs()
        d = 2.0 ** -19 * (1 + 20.0 * 5)  # |q| |k| scale is below 5 x 20 here
        assert ((out[:, h].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -13 + 4 * d) * mag).all()
        assert ((lse[:, h].double() - torch.logsumexp(z, 1)).abs() <= 2 * d + 2.0 ** -16).all()


def test_cached_many_sequences():
    """1,024 sequences, some without rows, some without positions."""
    g = np.random.default_rng(9)
    new = g.integers(0, 3, 1024)
    lens = np.maximum(g.integers(0, 40, 1024), new * g.integers(0, 2, 1024))
    c = Case(list(new), [int(x) for x in lens], 16, 1, 64, seed=10)
    c.check(2, 1)


# ------------------------------------------------------------- packed prompts


def _prompt(new, lens, heads, group, dim, block, seed=0, extra=3, scale=None, std=1.0, poke=None, same=False):
    g = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    koff = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    n, m = int(off[-1]) + extra, int(koff[-1]) + extra
    q = torch.from_numpy(std * g.standard_normal((n, heads * group, dim))).bfloat16()
    k, v = (torch.from_numpy(g.standard_normal((m, heads, dim))).bfloat16() for _ in range(2))
    k[koff[-1]:], v[koff[-1]:] = float("nan"), float("inf")
    if poke is not None:
        poke(q, k, v)
    want = R.prompt_attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), off, koff, block,
                              dim ** -0.5 if scale is None else scale)
    mark = torch.full((n, heads * group, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    out, lse = C.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), _ints(off), None if same else _ints(koff), block=block,
                                  scale=scale, lse=True, out=mark.clone())
    _close(out, want, off[-1], lse)
    assert torch.equal(out[off[-1]:], mark[off[-1]:])
    return out


@pytest.mark.parametrize("block", [0, 1, 8, 32])
@pytest.mark.parametrize("lens,heads,group,dim", [
    ([1], 1, 1, 64), ([1, 1, 1], 2, 8, 128), ([127], 1, 1, 128), ([128], 2, 2, 64), ([129, 3], 1, 4, 128),
    ([5, 0, 200, 33], 2, 8, 128), ([300], 1, 7, 64), ([257, 64], 1, 1, 128), ([90, 1], 3, 5, 128), ([70], 1, 64, 64),
    ([40, 41], 1, 33, 128),
])
def test_prompt_attention(lens, heads, group, dim, block):
    _prompt(lens, lens, heads, group, dim, block, seed=sum(lens) + group, same=True)


@pytest.mark.parametrize("block", [0, 1, 16])
@pytest.mark.parametrize("new,lens,heads,group,dim", [
    ([1], [500], 2, 8, 128), ([100, 3], [400, 130], 1, 4, 64), ([5, 9], [3, 0], 2, 2, 64), ([140], [129], 1, 2, 128),
    ([33, 0, 65], [1000, 20, 65], 2, 8, 128), ([20], [2000], 1, 16, 128),
])
def test_prompt_in_pieces(new, lens, heads, group, dim, block):
    """Fewer queries than keys, and more."""
    _prompt(new, lens, heads, group, dim, block, seed=sum(lens))


@pytest.mark.parametrize("what", ["k_nan", "v_nan", "v_inf", "q_nan", "k_inf"])
@pytest.mark.parametrize("at", [0, 60, 199])
def test_prompt_values_that_are_not_numbers(what, at):
    """They reach the queries that see them, and no others."""
    def poke(q, k, v):
        if what == "k_nan":
            k[at, 0, 3] = float("nan")
        elif what == "k_inf":  # the score of a query whose element is positive: +inf, whose softmax is NaN
            k[at, 0, 3] = float("inf")
            q[:, :, 3] = q[:, :, 3].abs() + 0.5
        elif what == "q_nan":
            q[at, 1, 0] = float("nan")
        else:
            v[at, 0, 5] = float("nan" if what == "v_nan" else "-inf")
    for heads, group in ((1, 2), (1, 16)):
        _prompt([200, 30], [200, 30], heads, group, 64, 1, seed=at, poke=poke)
        _prompt([200, 30], [200, 30], heads, group, 128, 16, seed=at, poke=poke)


def test_prompt_scores_of_minus_infinity():
    """Positions whose score is -inf have no weight; where all have, the row is empty."""
    def poke(q, k, v):
        q[:, :, 0] = 1.0
        k[:150, 0, 0] = float("-inf")
    q_ok = _prompt([200], [200], 1, 4, 64, 1, seed=2, poke=poke)
    assert not q_ok[:150].any() and q_ok[150:200].any()


@pytest.mark.parametrize("std,scale", [(30.0, None), (1.0, 50.0), (1e-3, 1e-3), (1e30, 1e-30), (1e-30, 1e29)])
def test_prompt_extreme_scores(std, scale):
    _prompt([300], [300], 1, 4, 128, 1, seed=11, std=std, scale=scale)


def _fp64(q, k, v, block, rows=512):
    """Results of one sequence in fp64 on the GPU, with the bound on their error."""
    n, Hq, D = q.shape
    L, H, _ = k.shape
    out, tol = torch.empty(q.shape, dtype=torch.float64, device=DEV), torch.empty(q.shape, dtype=torch.float64, device=DEV)
    for h in range(Hq):
        kk, vv = k[:, h // (Hq // H)].double(), v[:, h // (Hq // H)].double()
        for lo in range(0, n, rows):
            x = q[lo:lo + rows, h].double()
            p = L - n + torch.arange(lo, lo + x.shape[0], device=DEV)
            lim = torch.full_like(p, L) if block == 0 else torch.where(p < 0, 0, (p // block + 1) * block)
            z = x @ kk.T * D ** -0.5
            d = 2.0 ** -19 * (1 + (x.abs() @ kk.abs().T).amax(1, keepdim=True) * D ** -0.5)
            w = torch.softmax(z.masked_fill_(torch.arange(L, device=DEV) >= lim[:, None], -torch.inf), 1)
            o = w @ vv
            out[lo:lo + rows, h] = o
            tol[lo:lo + rows, h] = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -13 + 4 * d) * (w @ vv.abs())
    return out, tol


@pytest.mark.parametrize("new,length,heads,group,dim,block", [
    (4097, 4097, 2, 4, 128, 1), (1000, 9000, 1, 8, 128, 1), (3001, 3001, 2, 2, 64, 32), (2500, 2500, 1, 3, 64, 0),
    (128, 20011, 2, 8, 128, 1), (6000, 6000, 1, 1, 128, 1),
])
def test_prompt_long(new, length, heads, group, dim, block):
    g = torch.Generator(device=DEV).manual_seed(length)
    q = torch.randn((new, heads * group, dim), generator=g, device=DEV).bfloat16()
    k, v = (torch.randn((length, heads, dim), generator=g, device=DEV).bfloat16() for _ in range(2))
    out = C.prompt_attention(q, k, v, _ints([0, new]), _ints([0, length]), block=block)
    want, tol = _fp64(q, k, v, block)
    assert ((out.double() - want).abs() <= tol).all()


def test_prompt_strided_rows():
    """Slices of one projection, and head-major rows, give what contiguous rows give."""
    qkv = torch.randn(150, 8 + 2 + 2, 64, device=DEV).bfloat16()
    q, k, v = qkv.split((8, 2, 2), 1)
    off = _ints([0, 100, 150])
    want = C.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), off)
    assert torch.equal(C.prompt_attention(q, k, v, off), want)
    major = [t.permute(1, 0, 2).contiguous().permute(1, 0, 2) for t in (q, k, v)]
    assert torch.equal(C.prompt_attention(*major, off), want)


# --------------------------------------------------------------------- together


def _layer(cache, q, k, v, off, lens, table, koff):
    C.kv_write(cache, k, v, off, lens, table)
    a = C.kv_attention(q, cache, off, lens, table)
    kk, vv = C.kv_read(cache, koff, lens, table, int(sum(_layer.lens)))
    return a, C.prompt_attention(q, kk, vv, off, koff)


@pytest.mark.parametrize("group,dim", [(8, 128), (2, 64)])
def test_operations_together(group, dim):
    """Rows written and attended to from the cache, and the cache read back for the packed form: the same attention."""
    new, lens = [32, 5, 1, 60], [200, 5, 77, 60]
    c = Case(new, lens, 16, 2, dim, seed=12)
    off, ln, table = c.args()
    koff = _ints(np.concatenate([[0], np.cumsum(lens)]))
    _layer.lens = lens
    q = c.q(2 * group).to(DEV)
    k, v = (torch.randn(c.rows, 2, dim, device=DEV) for _ in range(2))
    cache = c.cache()
    a, b = _layer(cache, q, k, v, off, ln, table, koff)
    pages = R.write(c.pages, k.double().cpu().numpy(), v.double().cpu().numpy(), c.off, lens, c.table)
    assert np.array_equal(cache.pages.cpu().numpy(), pages)
    want = R.kv_attention(q.double().cpu().numpy(), pages, c.off, lens, c.table, 1, dim ** -0.5)
    _close(a, want, c.rows, cached=True)
    _close(b, want, c.rows)


def test_captured_and_replayed():
    """Two graphs with workspaces of their own, replayed with other lengths and rows than they were captured with."""
    c = Case([32, 1, 5], [300, 40, 9], 16, 2, 128, seed=13, spare=20, max_pages=30)
    c.table[:] = -1
    free = c.g.permutation(c.pages.shape[0])
    c.table[0, :len(free) // 2], c.table[1, :len(free) // 4] = free[:len(free) // 2], free[len(free) // 2:][:len(free) // 4]
    c.pages[..., 8 * 128:9 * 128] &= 0x37
    c.pages[..., 17 * 128:] &= 0x37
    off, ln, table = c.args()
    cache, q = c.cache(), c.q(16).to(DEV)
    k, v = (torch.randn(c.rows, 2, 128, device=DEV).bfloat16() for _ in range(2))
    koff, n_keys = _ints([0, 10, 20, 38]), 38
    runs = []
    for _ in range(2):
        ws = C.workspace(C.kv_attention_workspace_bytes(cache, c.rows, 16, *table.shape))
        ws2 = C.workspace(C.prompt_attention_workspace_bytes(c.rows, n_keys, 3, 16, 2, 128))
        out, out2 = torch.empty_like(q), torch.empty_like(q)

        def step(ws=ws, ws2=ws2, out=out, out2=out2):
            C.kv_write(cache, k, v, off, ln, table)
            C.kv_attention(q, cache, off, ln, table, ws=ws, out=out)
            kk, vv = C.kv_read(cache, koff, ln, table, n_keys)
            C.prompt_attention(q, kk, vv, off, koff, ws=ws2, out=out2)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        runs.append((graph, out, out2, ws, ws2, step))
    for lens, rows in (([300, 40, 9], [32, 1, 5]), ([35, 100, 0], [30, 3, 2]), ([200, 64, 3], [0, 38, 0])):
        off.copy_(_ints(np.concatenate([[0], np.cumsum(rows)])))
        ln.copy_(_ints(lens))
        for graph, *_ in runs:
            graph.replay()
        first = [t.clone() for t in runs[0][1:3]]
        for t in runs[1][1:3]:
            assert torch.equal(t, first[0] if t is runs[1][1] else first[1])
        runs[0][5]()
        assert torch.equal(runs[0][1], first[0]) and torch.equal(runs[0][2], first[1])
        for r in runs:
            C.workspace_status(r[3])
            C.workspace_status(r[4])


def test_one_workspace_for_calls_of_all_sizes():
    """Single tokens, blocks and prompts in turn through the same workspace."""
    cases = [Case([1], [5000], 32, 2, 128, seed=40), Case([32], [3000], 32, 2, 128, seed=41),
             Case([1] * 200, list(range(1, 201)), 16, 2, 128, seed=42), Case([2] * 90, list(range(2, 182, 2)), 16, 2, 128, seed=43)]
    calls = [(c.q(16).to(DEV), c.cache(), *c.args()) for c in cases]
    nbytes = max(C.kv_attention_workspace_bytes(a[1], a[0].shape[0], 16, *a[4].shape) for a in calls)
    k = torch.randn(32, 2, 128, device=DEV).bfloat16()
    nbytes = max(nbytes, C.prompt_attention_workspace_bytes(32, 32, 1, 16, 2, 128))
    ws = C.workspace(nbytes)
    want = [C.kv_attention(*a) for a in calls] + [C.prompt_attention(calls[1][0], k, k, calls[1][2])]
    for _ in range(3):
        for i in (0, 1, 2, 4, 0, 3, 1, 1, 0, 2):
            if i < 4:
                got = C.kv_attention(*calls[i], ws=ws)
            else:
                got = C.prompt_attention(calls[1][0], k, k, calls[1][2], ws=ws)
            assert torch.equal(got, want[i]), i
    C.workspace_status(ws)


@pytest.mark.parametrize("new,group", [(1, 8), (40, 8)])
def test_cached_queries_that_are_not_numbers(new, group):
    """A NaN or an infinity in a query stays in its row."""
    c = Case([new, 1], [200, 60], 16, 1, 64, seed=44)
    q = c.q(group)
    q[0, 1, 3], q[-1, 0, 5] = float("nan"), float("nan")
    want = R.kv_attention(q.double().numpy(), c.pages, c.off, c.lens, c.table, 1, 0.125)
    out, lse = C.kv_attention(q.to(DEV), c.cache(), *c.args(), lse=True)
    _close(out, want, c.rows, lse, cached=True)
    assert torch.isnan(out[0, 1]).all() and torch.isfinite(out[0, 0]).all()


@pytest.mark.parametrize("new,length,group", [(1, 70, 8), (1, 900, 8), (40, 200, 8), (40, 1500, 8)])
def test_cached_scores_of_minus_infinity(new, length, group):
    """A row whose scores are all -inf is empty, even where a value that it sees is NaN."""
    c = Case([new, 1], [length, 60], 16, 1, 64, seed=45)
    c.pages[:, :, :, 0:512:32] = c.pages[:, :, :, 0:512:32] & 0xF0 | 2  # element 0 of every key: 1 times its scale
    c.pages[c.table[0, 1], 0, 0, 17 * 64] = 0x7F
    q = c.q(group)
    q[0, 1] = 0.0
    q[0, 1, 0] = float("-inf")
    want = R.kv_attention(q.double().numpy(), c.pages, c.off, c.lens, c.table, 1, 0.125)
    assert not want[0][0, 1].any() and np.isnan(want[0][0, 0]).any()
    out, lse = C.kv_attention(q.to(DEV), c.cache(), *c.args(), lse=True)
    _close(out, want, c.rows, lse, cached=True)


def test_prompt_scores_of_minus_infinity_and_values_of_infinity():
    def poke(q, k, v):
        q[:, :, 0] = 1.0
        k[:150, 0, 0] = float("-inf")
        v[3, 0, 5], v[140, 0, 9] = float("inf"), float("nan")
    assert not _prompt([200], [200], 1, 4, 64, 1, seed=2, poke=poke)[:150].any()


@pytest.mark.parametrize("new,lens,heads,group,dim", [
    ([2], [500], 2, 8, 128), ([2], [70], 4, 8, 64), ([3], [300], 1, 5, 128),                   # tiles of 8 rows, few of them
    ([4, 4], [100, 333], 4, 8, 128), ([2, 2], [90, 40], 1, 16, 64), ([31, 1], [31, 64], 1, 2, 128),  # 32 rows each on average
    ([1] * 95, [40] * 95, 2, 4, 64), ([1] * 64, [33] * 64, 3, 16, 128), ([2] * 48, [60] * 48, 4, 8, 64),  # a piece for each warp
    ([1] * 94, [50] * 94, 2, 1, 128),
    ([0] * 90 + [250], [0] * 90 + [260], 1, 8, 64), ([1] * 60 + [130, 1], [20] * 60 + [400, 7], 2, 16, 64),  # one has most rows
])
def test_cached_attention_where_kernels_meet(new, lens, heads, group, dim):
    Case(new, lens, 16, heads, dim, seed=len(new)).check(heads * group, 1)


def test_no_pages_and_no_keys():
    """A table of no pages, keys and values without rows: every query sees nothing."""
    c = Case([3, 1], [3, 1], 16, 2, 64, seed=45)
    q = c.q(8).to(DEV)
    table = torch.zeros((2, 0), dtype=torch.int32, device=DEV)
    off, lens, _ = c.args()
    for rows in (4, 1):
        out, lse = C.kv_attention(q[:rows], c.cache(), off, lens, table, lse=True)
        assert not out.any() and (lse == -torch.inf).all()
    k, v = C.kv_read(c.cache(), off, lens, table, 4)
    assert not k.any() and not v.any()
    none = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    out, lse = C.prompt_attention(q, none, none, off, torch.zeros(3, dtype=torch.int32, device=DEV), lse=True)
    assert not out.any() and (lse == -torch.inf).all()


def test_streams_at_once():
    """Calls on three streams, each with its own workspace, give what they give alone."""
    cases = [Case([1, 32], [700, 300], 32, 2, 128, seed=20 + i) for i in range(3)]
    qs = [c.q(16).to(DEV) for c in cases]
    caches, args = [c.cache() for c in cases], [c.args() for c in cases]
    k = torch.randn(33, 2, 128, device=DEV).bfloat16()
    alone = [(C.kv_attention(q, cache, *a), C.prompt_attention(q, k, k, a[0])) for q, cache, a in zip(qs, caches, args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(5):
        for q, cache, a, s in zip(qs, caches, args, streams):
            s.wait_stream(torch.cuda.current_stream())
            got.append((C.kv_attention(q, cache, *a, stream=s), C.prompt_attention(q, k, k, a[0], stream=s)))
    torch.cuda.synchronize()
    for i, pair in enumerate(got):
        for x, y in zip(pair, alone[i % 3]):
            assert torch.equal(x, y)


def test_results_do_not_change_from_run_to_run():
    c = Case([1, 1, 32], [3000, 70, 900], 16, 2, 64, seed=30)
    q, cache, args = c.q(16).to(DEV), c.cache(), c.args()
    first = C.kv_attention(q, cache, *args, lse=True)
    ws = C.workspace(C.kv_attention_workspace_bytes(cache, c.rows, 16, *args[2].shape))
    for _ in range(20):
        again = C.kv_attention(q, cache, *args, lse=True, ws=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    C.workspace_status(ws)


def test_refusals_on_the_device():
    c = Case([1, 2], [30, 40], 16, 2, 64, seed=31)
    q, cache, (off, ln, table) = c.q(4).to(DEV), c.cache(), c.args()
    k = torch.zeros(3, 2, 64, device=DEV, dtype=torch.bfloat16)
    bad = [lambda: C.kv_attention(q.float(), cache, off, ln, table), lambda: C.kv_attention(q[:, :3], cache, off, ln, table),
           lambda: C.kv_attention(q[..., :32], cache, off, ln, table), lambda: C.kv_attention(q, cache, off[:2], ln, table),
           lambda: C.kv_attention(q, cache, off, ln.long(), table), lambda: C.kv_attention(q, cache, off, ln, table[:, ::2]),
           lambda: C.kv_attention(q, cache, off, ln, table, scale=0.0), lambda: C.kv_attention(q, cache, off, ln, table, block=-1),
           lambda: C.kv_attention(q, cache, off, ln, table, block=1 << 32),
           lambda: C.kv_attention(q, cache, off, ln, table, out=q.float()),
           lambda: C.kv_attention(q, cache, off, ln, table, lse=torch.zeros(3, 3, device=DEV)),
           lambda: C.kv_attention(q, cache, off, ln, table, ws=torch.zeros(8, dtype=torch.uint8, device=DEV)),
           lambda: C.kv_attention(q, cache, off.cpu(), ln, table), lambda: C.kv_write(cache, k, k.float(), off, ln, table),
           lambda: C.kv_write(cache, k[:2], k, off, ln, table), lambda: C.kv_write(cache, k[:, :1], k, off, ln, table),
           lambda: C.kv_read(cache, off, ln, table, -1), lambda: C.kv_read(cache, off, ln, table, 3, out=(k, k[:2])),
           lambda: C.prompt_attention(q, k, k[:2], off), lambda: C.prompt_attention(q, k[:, :1], k, off),
           lambda: C.prompt_attention(q, k, k, off, off[:2]), lambda: C.prompt_attention(q.half(), k, k, off),
           lambda: C.prompt_attention(q[0], k, k, off), lambda: C.prompt_attention(q, k.expand(3, 2, 64)[:, :1].expand(3, 2, 64), k, off)]
    for i, f in enumerate(bad):
        with pytest.raises(C.CloverError):
            f()
    assert C.kv_attention(q[:0], cache, off, ln, table).shape == (0, 4, 64)
    assert C.prompt_attention(q[:0], k, k, off).shape == (0, 4, 64)
