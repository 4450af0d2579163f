"""The attention operations on the host: what the library and its binding
refuse before anything is enqueued (no call here reaches a GPU), their size
queries, and pins of the oracle the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from block_diffusion_moe_gb300 import build as B
from block_diffusion_moe_gb300 import clover as C
from oracle import attention as R


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.lib()


CACHE = dict(pages=0x10000, n_pages=10, page_tokens=32, kv_heads=2, head_dim=128, k_exp=0, v_exp=0)
SEQS = dict(offsets=0x20000, lens=0x30000, table=0x40000, n_seqs=3, max_pages=5)
ROWS = dict(data=0x100000, row_stride=2048, head_stride=128)


def _cache(**kw):
    return C.KvCacheArgs(*dict(CACHE, **kw).values())


def _seqs(**kw):
    return C.KvSeqs(*dict(SEQS, **kw).values())


def _rows(**kw):
    return C.Rows(*dict(ROWS, **kw).values())


def _write(lib, cache=None, seqs=None, k=None, v=None, type=1, n=7):
    return lib.clover_kv_write(cache or _cache(), seqs or _seqs(), k or _rows(), v or _rows(), type, n, None)


def _read(lib, cache=None, seqs=None, k=0x100000, v=0x200000, n=7):
    return lib.clover_kv_read(cache or _cache(), seqs or _seqs(), k, v, n, None)


def _cached(lib, cache=None, seqs=None, q=None, n=7, heads=16, scale=0.1, block=1, out=0x200000, lse=None, ws=0x300000,
            nbytes=1 << 30):
    return lib.clover_kv_attention(cache or _cache(), seqs or _seqs(), q or _rows(), n, heads, scale, block, out, lse, ws,
                                   nbytes, None)


def _prompt(lib, offsets=0x20000, k_offsets=0x30000, n_seqs=3, q=None, k=None, v=None, n=7, keys=9, heads=16, kv_heads=2,
            dim=128, scale=0.1, block=1, out=0x200000, lse=None, ws=0x300000, nbytes=1 << 30):
    return lib.clover_prompt_attention(C.PromptSeqs(offsets, k_offsets, n_seqs), q or _rows(), k or _rows(), v or _rows(), n,
                                       keys, heads, kv_heads, dim, scale, block, out, lse, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(page_tokens=0), C.ERR_UNSUPPORTED_SHAPE), (dict(page_tokens=24), C.ERR_UNSUPPORTED_SHAPE),
    (dict(page_tokens=65552), C.ERR_UNSUPPORTED_SHAPE), (dict(kv_heads=0), C.ERR_UNSUPPORTED_SHAPE),
    (dict(kv_heads=257), C.ERR_UNSUPPORTED_SHAPE), (dict(head_dim=96), C.ERR_UNSUPPORTED_SHAPE),
    (dict(head_dim=256), C.ERR_UNSUPPORTED_SHAPE), (dict(n_pages=0), C.ERR_UNSUPPORTED_SHAPE),
    (dict(k_exp=65), C.ERR_INVALID_ARG), (dict(v_exp=-65), C.ERR_INVALID_ARG), (dict(pages=None), C.ERR_INVALID_ARG),
    (dict(pages=0x10008), C.ERR_INVALID_ARG),
])
def test_cache_refused(lib, kw, code):
    for f in (_write, _read, _cached):
        assert f(lib, cache=_cache(**kw)) == code, f
        assert C.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), C.ERR_UNSUPPORTED_SHAPE), (dict(n_seqs=1025), C.ERR_UNSUPPORTED_SHAPE),
    (dict(max_pages=-1), C.ERR_UNSUPPORTED_SHAPE), (dict(max_pages=(1 << 19) + 1), C.ERR_UNSUPPORTED_SHAPE),
    (dict(offsets=None), C.ERR_INVALID_ARG), (dict(lens=None), C.ERR_INVALID_ARG), (dict(table=None), C.ERR_INVALID_ARG),
    (dict(offsets=0x20002), C.ERR_INVALID_ARG), (dict(lens=0x30001), C.ERR_INVALID_ARG),
    (dict(table=0x40002), C.ERR_INVALID_ARG),
])
def test_sequences_refused(lib, kw, code):
    for f in (_write, _read, _cached):
        assert f(lib, seqs=_seqs(**kw)) == code, f


@pytest.mark.parametrize("kw", [dict(data=None), dict(data=0x100008), dict(row_stride=127), dict(row_stride=2049),
                                dict(head_stride=64), dict(head_stride=129), dict(row_stride=1 << 37)])
def test_rows_refused(lib, kw):
    bad = _rows(**kw)
    for rc in (_write(lib, k=bad), _write(lib, v=bad), _cached(lib, q=bad), _prompt(lib, q=bad), _prompt(lib, k=bad),
               _prompt(lib, v=bad)):
        assert rc == C.ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), C.ERR_UNSUPPORTED_SHAPE), (dict(n=(1 << 24) + 1), C.ERR_UNSUPPORTED_SHAPE),
    (dict(heads=0), C.ERR_UNSUPPORTED_SHAPE), (dict(heads=15), C.ERR_UNSUPPORTED_SHAPE),
    (dict(heads=130), C.ERR_UNSUPPORTED_SHAPE), (dict(scale=0.0), C.ERR_INVALID_ARG),
    (dict(scale=-1.0), C.ERR_INVALID_ARG), (dict(scale=float("nan")), C.ERR_INVALID_ARG),
    (dict(scale=float("inf")), C.ERR_INVALID_ARG), (dict(block=-1), C.ERR_INVALID_ARG), (dict(out=None), C.ERR_INVALID_ARG),
    (dict(out=0x200008), C.ERR_INVALID_ARG), (dict(lse=0x400002), C.ERR_INVALID_ARG), (dict(ws=None), C.ERR_INVALID_ARG),
    (dict(ws=0x300010), C.ERR_INVALID_ARG), (dict(nbytes=100), C.ERR_WORKSPACE_TOO_SMALL),
])
def test_attention_arguments_refused(lib, kw, code):
    for f in (_cached, _prompt):
        assert f(lib, **kw) == code, f
        assert C.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(offsets=None), C.ERR_INVALID_ARG), (dict(k_offsets=None), C.ERR_INVALID_ARG),
    (dict(offsets=0x20001), C.ERR_INVALID_ARG), (dict(k_offsets=0x30002), C.ERR_INVALID_ARG),
    (dict(n_seqs=0), C.ERR_UNSUPPORTED_SHAPE), (dict(n_seqs=1025), C.ERR_UNSUPPORTED_SHAPE),
    (dict(keys=-1), C.ERR_UNSUPPORTED_SHAPE), (dict(keys=(1 << 24) + 1), C.ERR_UNSUPPORTED_SHAPE),
    (dict(dim=32), C.ERR_UNSUPPORTED_SHAPE), (dict(kv_heads=0), C.ERR_UNSUPPORTED_SHAPE),
])
def test_prompt_arguments_refused(lib, kw, code):
    assert _prompt(lib, **kw) == code


def test_copies_refused(lib):
    assert _write(lib, type=2) == C.ERR_INVALID_ARG
    assert _write(lib, n=-1) == C.ERR_UNSUPPORTED_SHAPE
    assert _read(lib, n=-1) == C.ERR_UNSUPPORTED_SHAPE
    assert _read(lib, k=None) == C.ERR_INVALID_ARG
    assert _read(lib, v=0x200008) == C.ERR_INVALID_ARG
    assert lib.clover_kv_write(None, _seqs(), _rows(), _rows(), 1, 7, None) == C.ERR_INVALID_ARG
    assert lib.clover_kv_read(_cache(), None, 0x100000, 0x200000, 7, None) == C.ERR_INVALID_ARG


def test_nothing_to_do(lib):
    none = C.Rows(None, 0, 0)
    empty, seqs = _cache(pages=None), _seqs(offsets=None, lens=None, table=None)
    assert _write(lib, empty, seqs, none, none, n=0) == C.OK
    assert _read(lib, empty, seqs, None, None, n=0) == C.OK
    assert _cached(lib, empty, seqs, none, n=0, out=None) == C.OK
    assert _prompt(lib, offsets=None, k_offsets=None, q=none, k=none, v=none, n=0, out=None) == C.OK


def test_sizes(lib):
    assert lib.clover_kv_page_bytes(64, 2, 128) == 64 * 2 * 144
    assert lib.clover_kv_page_bytes(16, 1, 64) == 16 * 72
    for bad in ((8, 1, 64), (16, 0, 64), (16, 1, 80)):
        assert lib.clover_kv_page_bytes(*bad) == 0
    f, g = lib.clover_kv_attention_workspace_bytes, lib.clover_prompt_attention_workspace_bytes
    assert f(_cache(pages=None), 0, 16, 1, 0) > 0 and g(0, 0, 1, 16, 2, 128) > 0
    assert f(_cache(), 1, 15, 1, 1) == 0 and f(_cache(), 1, 16, 0, 1) == 0 and f(None, 1, 16, 1, 1) == 0
    assert g(1, 1, 1, 15, 2, 128) == 0 and g(1, 1, 0, 16, 2, 128) == 0 and g(-1, 1, 1, 16, 2, 128) == 0


@pytest.mark.parametrize("heads,kv_heads,dim", [(16, 2, 128), (32, 8, 64), (7, 1, 128), (64, 1, 64), (5, 5, 128)])
def test_workspaces_cover_fewer_rows(lib, heads, kv_heads, dim):
    """A workspace for so many rows (and keys) serves every call of fewer."""
    rows = list(range(0, 700)) + list(range(700, 70000, 1013))
    for n_seqs in (1, 3, 64, 1024):
        for pages in (0, 1, 7, 64, 4096):
            c = _cache(kv_heads=kv_heads, head_dim=dim)
            sizes = [lib.clover_kv_attention_workspace_bytes(c, n, heads, n_seqs, pages) for n in rows]
            assert sizes[0] >= 256 and all(a <= b for a, b in zip(sizes, sizes[1:]))
            sizes = [lib.clover_prompt_attention_workspace_bytes(n, pages * 64, n_seqs, heads, kv_heads, dim) for n in rows]
            assert sizes[0] >= 256 and all(a <= b for a, b in zip(sizes, sizes[1:]))
        for n in (1, 33, 4000):
            c = _cache(kv_heads=kv_heads, head_dim=dim)
            sizes = [lib.clover_kv_attention_workspace_bytes(c, n, heads, n_seqs, p) for p in range(0, 5000, 7)]
            assert all(a <= b for a, b in zip(sizes, sizes[1:]))
            sizes = [lib.clover_prompt_attention_workspace_bytes(n, p, n_seqs, heads, kv_heads, dim)
                     for p in range(0, 200000, 333)]
            assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_cache_tensor_is_checked(lib):
    pages = torch.zeros((4, 2, 2, 18 * 64), dtype=torch.uint8)
    c = C.KvCache(pages, k_exp=-3)
    assert (c.n_pages, c.kv_heads, c.page_tokens, c.head_dim, c.k_exp, c.v_exp) == (4, 2, 32, 64, -3, 0)
    assert c.pages is pages
    with pytest.raises(AttributeError):
        c.pages = pages
    bad = [lambda: C.KvCache(pages.int()), lambda: C.KvCache(pages[0]), lambda: C.KvCache(pages[:, :, :, :-18]),
           lambda: C.KvCache(torch.zeros((4, 2, 2, 100), dtype=torch.uint8)), lambda: C.KvCache(pages[:0]),
           lambda: C.KvCache(pages, k_exp=65), lambda: C.KvCache(pages, v_exp=1 << 40),
           lambda: C.KvCache.empty(4, 24, 2, 64, device="cpu"), lambda: C.KvCache.empty(4, 32, 2, 80, device="cpu"),
           lambda: C.KvCache(torch.zeros((4, 2, 2, 18 * 80), dtype=torch.uint8))]
    for f in bad:
        with pytest.raises(C.CloverError):
            f()
    e = C.KvCache.empty(3, 48, 1, 128, device="cpu")
    assert e.pages.shape == (3, 1, 3, 2304) and not e.pages.any()


def test_wrappers_refuse_host_tensors(lib):
    c = C.KvCache(torch.zeros((4, 2, 2, 18 * 64), dtype=torch.uint8))
    i, q = torch.zeros(2, dtype=torch.int32), torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    k, table = torch.zeros((1, 2, 64), dtype=torch.bfloat16), torch.zeros((1, 1), dtype=torch.int32)
    for f in (lambda: C.kv_write(c, k, k, i, i[:1], table), lambda: C.kv_read(c, i, i[:1], table, 1),
              lambda: C.kv_attention(q, c, i, i[:1], table), lambda: C.prompt_attention(q, k, k, i)):
        with pytest.raises(C.CloverError):
            f()
    with pytest.raises(C.CloverError):
        C.kv_attention_workspace_bytes(c, 1 << 40, 4, 1, 1)
    with pytest.raises(C.CloverError):
        C.prompt_attention_workspace_bytes(1, 1 << 33, 1, 4, 2, 64)


# ----------------------------------------------------------------- oracle pins


def test_oracle_quantises_by_hand():
    x = np.zeros(16)
    x[:6] = [6.0, -3.0, 0.25, 0.75, 5.0, -0.2]  # scale 1: ties go to the even code
    codes, scales = R.quantize_row(x, 0)
    assert R.E4M3[scales[0]] == 1.0
    assert list(R.decode_row(codes, scales, 0)[:6]) == [6.0, -3.0, 0.0, 1.0, 4.0, 0.0]
    x[0] = np.inf
    assert np.isnan(R.decode_row(*R.quantize_row(x, 0), 0)).all()
    assert list(R.decode_row(*R.quantize_row(np.full(16, 12.0), 1), 1)) == [12.0] * 16


def test_oracle_write_and_positions_round_trip():
    rng = np.random.default_rng(0)
    pages = rng.integers(0, 256, (5, 2, 2, 18 * 64)).astype(np.uint8)
    k, v = rng.standard_normal((2, 40, 2, 64)).astype(np.float32)
    table = np.array([[3, 1, -1], [0, 9, 4]])
    after = R.write(pages, k, v, np.array([0, 38, 39]), np.array([38, 1]), table)
    kk, vv, there = R.positions(after, table[0], 38)
    assert there.all()
    assert np.abs(kk - k[:38]).max() < 1.0 and np.abs(vv - v[:38]).max() < 1.0
    assert (after[2] == pages[2]).all() and (after[4] == pages[4]).all()
    _, _, there = R.positions(after, table[1], 65)
    assert there[:32].all() and not there[32:64].any() and there[64]


def test_oracle_attention_by_hand():
    q = np.zeros((2, 2, 64))
    k, v = np.zeros((3, 1, 64)), np.zeros((3, 1, 64))
    v[:, 0, 0] = [1.0, 2.0, 6.0]
    out, lse, *_ = R.attend(q, k, v, np.ones(3, dtype=bool), 1, 1.0)
    assert np.allclose(out[:, :, 0], [[1.5, 1.5], [3.0, 3.0]]) and np.allclose(np.exp(lse), [[2, 2], [3, 3]])
    out, *_ = R.attend(q, k, v, np.array([True, False, True]), 0, 1.0)
    assert np.allclose(out[:, :, 0], 3.5)
    out, lse, *_ = R.attend(np.zeros((5, 2, 64)), k, v, np.ones(3, dtype=bool), 2, 1.0)
    assert (out[:2] == 0).all() and (lse[:2] == -np.inf).all()  # before the first position
    assert np.allclose(out[2:, 0, 0], [1.5, 1.5, 3.0])


@pytest.mark.parametrize("block", [0, 1, 2, 5])
def test_oracle_visibility(block):
    """A query sees exactly the positions whose change changes its result."""
    rng = np.random.default_rng(block)
    q, k, v = rng.standard_normal((4, 1, 64)), rng.standard_normal((7, 1, 64)), rng.standard_normal((7, 1, 64))
    base = R.attend(q, k, v, np.ones(7, dtype=bool), block, 0.125)[0]
    for j in range(7):
        w = v.copy()
        w[j] += 1.0
        moved = (R.attend(q, k, w, np.ones(7, dtype=bool), block, 0.125)[0] != base).any((1, 2))
        assert list(moved) == [j < R.limit(3 + i, 7, block) for i in range(4)]


def test_struct_sizes():
    assert ctypes.sizeof(C.KvCacheArgs) == 32 and ctypes.sizeof(C.KvSeqs) == 32
    assert ctypes.sizeof(C.PromptSeqs) == 24 and ctypes.sizeof(C.Rows) == 24


def test_shared_status_arguments(lib):
    assert lib.clover_attention_shared_status(None) == C.ERR_INVALID_ARG
