"""Attention on tiles where a CTA has several items (pairs of tiles of 128 rows): two, nine and twenty, more than are
worked out at a CTA's beginning, on the GPU."""
import numpy as np
import pytest
import torch

from block_diffusion_moe_gb300 import clover as C
from tests.test_gpu_attention import DEV, _ints

pytestmark = pytest.mark.gpu

GROUP = 64  # two tokens a tile: many items of few rows


def _sequences(per_cta, heads):
    """Rows and lengths of five sequences, one empty, one with more rows than positions: so many items for each SM, and a few."""
    n = 4 * per_cta * torch.cuda.get_device_properties(0).multi_processor_count // heads
    new = [n // 2 + 3, 1, 0, n - n // 2, 6]
    return new, [new[0], 8, 3, new[3] + 130, 4]


def _expected(q, k, v, block, half_step, rows=1024):
    """One sequence in fp64: out, its bound, lse, its bound. Scores, sums and the result are given what they are given in the
    shorter tests (test_gpu_attention), numerators their own half step."""
    n, L = q.shape[0], k.shape[0]
    res = [torch.zeros(q.shape, dtype=torch.float64, device=DEV) for _ in range(2)]
    res += [torch.full(q.shape[:2], -torch.inf, dtype=torch.float64, device=DEV), torch.zeros(q.shape[:2], dtype=torch.float64, device=DEV)]
    for h in range(q.shape[1]):
        kk, vv = k[:, h // GROUP].double(), v[:, h // GROUP].double()
        for lo in range(0, n, rows):
            at = slice(lo, min(lo + rows, n))
            x = q[at, h].double()
            p = L - n + torch.arange(at.start, at.stop, device=DEV)
            lim = torch.full_like(p, L) if block == 0 else torch.where(p < 0, 0, (p // block + 1) * block)
            see = torch.arange(L, device=DEV) < lim[:, None]
            z = (x @ kk.T * x.shape[1] ** -0.5).masked_fill_(~see, -torch.inf)
            d = 2.0 ** -19 * (1 + (x.abs() @ kk.abs().T).amax(1) * x.shape[1] ** -0.5)
            w = torch.softmax(z, 1).nan_to_num(0.0)
            o = w @ vv
            res[0][at, h] = o
            res[1][at, h] = 2.0 ** -8 * o.abs() + (half_step + 2.0 ** -13 + 4 * d[:, None]) * (w @ vv.abs()) + 2.0 ** -36 * vv.abs().sum(0)
            res[2][at, h] = torch.logsumexp(z, 1)
            res[3][at, h] = 2 * d + 2.0 ** -20 * res[2][at, h].abs().nan_to_num(posinf=0.0)
    return res


def _check(got, at, want):
    out, tol, lse, lse_tol = want
    err = (got[0][at].double() - out).abs()
    assert (err <= tol).all(), (err / tol).max()
    z = got[1][at].double()
    assert ((z == lse) | ((z - lse).abs() <= lse_tol)).all()


@pytest.mark.parametrize("per_cta,heads,dim,block", [(2, 2, 128, 1), (2, 1, 64, 32), (9, 1, 128, 32), (9, 2, 64, 0), (20, 1, 64, 1)])
def test_prompt_items(per_cta, heads, dim, block):
    new, lens = _sequences(per_cta, heads)
    g = torch.Generator(device=DEV).manual_seed(per_cta)
    off, koff = (np.concatenate([[0], np.cumsum(x)]) for x in (new, lens))
    q = torch.randn((int(off[-1]) + 3, heads * GROUP, dim), generator=g, device=DEV).bfloat16()
    k, v = (torch.randn((int(koff[-1]) + 3, heads, dim), generator=g, device=DEV).bfloat16() for _ in range(2))
    ws = C.workspace(C.prompt_attention_workspace_bytes(q.shape[0], k.shape[0], len(new), heads * GROUP, heads, dim))
    mark = torch.full_like(q, 7.0)
    got = C.prompt_attention(q, k, v, _ints(off), _ints(koff), block=block, lse=True, out=mark, ws=ws)
    C.workspace_status(ws)
    assert mark[int(off[-1]):].eq(7.0).all()
    for s in range(len(new)):
        at, keys = slice(off[s], off[s + 1]), slice(koff[s], koff[s + 1])
        _check(got, at, _expected(q[at], k[keys], v[keys], block, 2.0 ** -8))


@pytest.mark.parametrize("per_cta,heads,dim,block", [(2, 2, 128, 1), (2, 1, 64, 32), (9, 1, 128, 32), (9, 2, 64, 0), (20, 1, 64, 1)])
def test_cached_items(per_cta, heads, dim, block):
    new, lens = _sequences(per_cta, heads)
    g = torch.Generator(device=DEV).manual_seed(per_cta + 1)
    off, koff = (np.concatenate([[0], np.cumsum(x)]) for x in (new, lens))
    used = [-(-L // 32) for L in lens]
    cache = C.KvCache.empty(sum(used), 32, heads, dim)
    table = torch.full((len(new), max(used)), -1, dtype=torch.int32, device=DEV)
    ids = torch.randperm(sum(used), generator=g, device=DEV).int()
    for s, u in enumerate(used):
        table[s, :u] = ids[sum(used[:s]):sum(used[:s]) + u]
    k, v = (torch.randn((int(koff[-1]), heads, dim), generator=g, device=DEV).bfloat16() for _ in range(2))
    C.kv_write(cache, k, v, _ints(koff), _ints(lens), table)
    k, v = C.kv_read(cache, _ints(koff), _ints(lens), table, int(koff[-1]))
    q = torch.randn((int(off[-1]) + 3, heads * GROUP, dim), generator=g, device=DEV).bfloat16()
    ws = C.workspace(C.kv_attention_workspace_bytes(cache, q.shape[0], heads * GROUP, *table.shape))
    mark = torch.full_like(q, 7.0)
    got = C.kv_attention(q, cache, _ints(off), _ints(lens), table, block=block, lse=True, out=mark, ws=ws)
    C.workspace_status(ws)
    assert mark[int(off[-1]):].eq(7.0).all()
    for s in range(len(new)):
        at, keys = slice(off[s], off[s + 1]), slice(koff[s], koff[s + 1])
        _check(got, at, _expected(q[at], k[keys], v[keys], block, 2.0 ** -12))


@pytest.mark.parametrize("cached", [False, True])
def test_odd_values_of_some_items(cached):
    """1,024 sequences of three items each; the last position's value of every third sequence is not a number in places. It
    changes those sequences' last row there, and no other."""
    n, L, dim = 1024, 12, 64
    g = torch.Generator(device=DEV).manual_seed(7)
    off = _ints(np.arange(n + 1) * L)
    q = torch.randn((n * L, GROUP, dim), generator=g, device=DEV).bfloat16()
    k, v = (torch.randn((n * L, 1, dim), generator=g, device=DEV).bfloat16() for _ in range(2))
    last = torch.arange(n, device=DEV)[::3] * L + L - 1
    lens, table = _ints([L] * n), torch.arange(n, device=DEV, dtype=torch.int32)[:, None].contiguous()
    cache = C.KvCache.empty(n, 16, 1, dim)

    def call():
        if not cached:
            return C.prompt_attention(q, k, v, off, lse=True)
        C.kv_write(cache, k, v, off, lens, table)
        return C.kv_attention(q, cache, off, lens, table, lse=True)

    first = call()
    v[last, 0, 20] = float("nan")
    again = call()
    C.attention_status()
    changed = torch.zeros(first[0].shape, dtype=torch.bool, device=DEV)
    if cached:
        changed[last, :, 16:32] = True  # (its block of 16)
    else:
        changed[last, :, 20] = True
    assert again[0][changed].isnan().all() and not first[0].isnan().any()
    assert torch.equal(again[0][~changed], first[0][~changed]) and torch.equal(again[1], first[1])
