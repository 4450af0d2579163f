"""The routed-expert operations on the host: what the library refuses before
it enqueues anything (no call here reaches a GPU), its size queries, and pins
of the oracle the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from block_diffusion_moe_gb300 import build as B
from block_diffusion_moe_gb300 import clover as C
from oracle import moe_ops as R


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.lib()


def _routing(**kw):
    base = dict(n_experts=256, top_k=8, score="softmax", n_groups=8, top_groups=4, group_rank=2)
    base.update(kw)
    return C.make_routing(**base)


ROUTE = dict(logits=0x10000, type=0, ld=256, bias=0x20000, M=32, idx=0x30000, w=0x40000, offsets=0x50000, rows=0x60000,
             pos=0x70000, ws=0x100000, nbytes=1 << 24, stream=None)


def _route(lib, r, **kw):
    a = dict(ROUTE, **kw)
    return lib.clover_route(r, *a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(n_experts=0), C.ERR_UNSUPPORTED_SHAPE), (dict(n_experts=513, n_groups=1, top_groups=1), C.ERR_UNSUPPORTED_SHAPE),
    (dict(top_k=0), C.ERR_UNSUPPORTED_SHAPE), (dict(top_k=33), C.ERR_UNSUPPORTED_SHAPE),
    (dict(n_experts=4, n_groups=1, top_groups=1, top_k=5), C.ERR_UNSUPPORTED_SHAPE),
    (dict(n_groups=7), C.ERR_UNSUPPORTED_SHAPE), (dict(n_groups=64, top_groups=4), C.ERR_UNSUPPORTED_SHAPE),
    (dict(n_groups=0), C.ERR_UNSUPPORTED_SHAPE), (dict(top_groups=9), C.ERR_INVALID_ARG),
    (dict(top_groups=0), C.ERR_INVALID_ARG), (dict(group_rank=3), C.ERR_INVALID_ARG),
    (dict(scale=float("nan")), C.ERR_INVALID_ARG), (dict(scale=float("inf")), C.ERR_INVALID_ARG),
])
def test_route_rules_refused(lib, kw, code):
    r = _routing(**kw)
    assert _route(lib, r) == code
    assert C.last_error()
    assert lib.clover_route_workspace_bytes(r, 32) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), C.ERR_INVALID_ARG), (dict(idx=None), C.ERR_INVALID_ARG), (dict(w=None), C.ERR_INVALID_ARG),
    (dict(type=2), C.ERR_INVALID_ARG), (dict(ld=255), C.ERR_INVALID_ARG), (dict(logits=0x10002), C.ERR_INVALID_ARG),
    (dict(type=1, logits=0x10001), C.ERR_INVALID_ARG), (dict(rows=None), C.ERR_INVALID_ARG),
    (dict(offsets=None), C.ERR_INVALID_ARG), (dict(pos=0x70002), C.ERR_INVALID_ARG), (dict(M=-1), C.ERR_UNSUPPORTED_SHAPE),
    (dict(M=1 << 28), C.ERR_UNSUPPORTED_SHAPE), (dict(ws=None), C.ERR_INVALID_ARG), (dict(ws=0x100010), C.ERR_INVALID_ARG),
    (dict(nbytes=1000), C.ERR_WORKSPACE_TOO_SMALL),
])
def test_route_arguments_refused(lib, kw, code):
    assert _route(lib, _routing(), **kw) == code
    assert C.last_error()


def test_route_workspace_covers_fewer_tokens(lib):
    """A workspace for max_tokens serves every call of fewer tokens."""
    r = _routing()
    sizes = [lib.clover_route_workspace_bytes(r, m) for m in range(0, 40000, 37)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert lib.clover_route_workspace_bytes(r, -1) == 0
    assert lib.clover_route_workspace_bytes(r, 1 << 28) == 0


def test_score_name_refused():
    with pytest.raises(C.CloverError):
        C.make_routing(8, 2, score="relu")


QUANT = dict(fmt=0, x=0x10000, type=1, ldx=256, mats=2, rows=10, cols=256, exp=0, codes=0x20000, scales=0x30000, stream=None)
ROWS = dict(fmt=0, x=0x10000, type=1, ldx=256, n_src=10, cols=256, exp=0, src=0x40000, div=8, n_rows=10, offsets=0x50000,
            groups=4, codes=0x20000, scales=0x30000, stream=None)
DEQ = dict(fmt=0, codes=0x20000, scales=0x30000, mats=1, rows=10, cols=256, exp=0, offsets=0x50000, groups=4, out=0x60000,
           stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), C.ERR_INVALID_ARG), (dict(cols=96), C.ERR_UNSUPPORTED_SHAPE), (dict(cols=0), C.ERR_UNSUPPORTED_SHAPE),
    (dict(cols=(1 << 20) + 64), C.ERR_UNSUPPORTED_SHAPE), (dict(exp=65), C.ERR_INVALID_ARG), (dict(exp=-65), C.ERR_INVALID_ARG),
    (dict(codes=None), C.ERR_INVALID_ARG), (dict(scales=0x30008), C.ERR_INVALID_ARG),
])
def test_fp4_arguments_refused(lib, kw, code):
    for f, base in ((lib.clover_quantize_fp4, QUANT), (lib.clover_quantize_fp4_rows, ROWS), (lib.clover_dequantize_fp4, DEQ)):
        assert f(*dict(base, **kw).values()) == code, f
        assert C.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), C.ERR_INVALID_ARG), (dict(x=0x10008), C.ERR_INVALID_ARG), (dict(type=2), C.ERR_INVALID_ARG),
    (dict(ldx=255), C.ERR_INVALID_ARG), (dict(ldx=257), C.ERR_INVALID_ARG),
])
def test_fp4_input_refused(lib, kw, code):
    for f, base in ((lib.clover_quantize_fp4, QUANT), (lib.clover_quantize_fp4_rows, ROWS)):
        assert f(*dict(base, **kw).values()) == code, f


def test_fp4_groups_refused(lib):
    for f, base in ((lib.clover_quantize_fp4_rows, ROWS), (lib.clover_dequantize_fp4, DEQ)):
        assert f(*dict(base, groups=0).values()) == C.ERR_UNSUPPORTED_SHAPE
        assert f(*dict(base, groups=513).values()) == C.ERR_UNSUPPORTED_SHAPE
        assert f(*dict(base, offsets=0x50002).values()) == C.ERR_INVALID_ARG
    f = lib.clover_quantize_fp4_rows
    assert f(*dict(ROWS, offsets=None).values()) == C.ERR_INVALID_ARG
    assert f(*dict(ROWS, src=0x40002).values()) == C.ERR_INVALID_ARG
    assert f(*dict(ROWS, div=0).values()) == C.ERR_INVALID_ARG
    assert f(*dict(ROWS, n_src=-1).values()) == C.ERR_INVALID_ARG
    assert f(*dict(ROWS, n_rows=-1).values()) == C.ERR_UNSUPPORTED_SHAPE
    assert lib.clover_dequantize_fp4(*dict(DEQ, mats=2).values()) == C.ERR_INVALID_ARG
    assert lib.clover_dequantize_fp4(*dict(DEQ, out=None).values()) == C.ERR_INVALID_ARG
    assert lib.clover_quantize_fp4(*dict(QUANT, mats=1 << 20, rows=1 << 12).values()) == C.ERR_UNSUPPORTED_SHAPE
    assert lib.clover_quantize_fp4(*dict(QUANT, rows=-1).values()) == C.ERR_INVALID_ARG
    # nothing to do: no data pointers needed
    assert f(*dict(ROWS, n_rows=0, x=None, codes=None, offsets=None).values()) == C.OK
    assert lib.clover_quantize_fp4(*dict(QUANT, rows=0, x=None).values()) == C.OK
    assert lib.clover_dequantize_fp4(*dict(DEQ, rows=0, out=None).values()) == C.OK


def test_fp4_scale_bytes(lib):
    f, g = lib.clover_fp4_scale_bytes, lib.clover_fp4_grouped_scale_bytes
    assert f(0, 3, 129, 64) == 3 * 2 * 1 * 512
    assert f(0, 1, 128, 2048) == 32 * 512
    assert f(1, 1, 128, 2048) == 16 * 512
    assert f(1, 1, 1, 64) == 512
    assert f(0, 1, 0, 64) == 0 and f(0, 1, 1, 65) == 0 and f(5, 1, 1, 64) == 0
    assert g(0, 256, 7, 64) == (2 + 7) * 512
    assert g(1, 1000, 1, 192) == (7 + 1) * 2 * 512
    assert g(0, 1, 0, 64) == 0


COMBINE = dict(y=0x10000, n_rows=256, pos=0x20000, w=0x30000, shared=None, x=0x40000, out=0x80000, M=32, K=8, H=256,
               stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(y=None), C.ERR_INVALID_ARG), (dict(pos=None), C.ERR_INVALID_ARG), (dict(w=None), C.ERR_INVALID_ARG),
    (dict(out=None), C.ERR_INVALID_ARG), (dict(y=0x10008), C.ERR_INVALID_ARG), (dict(shared=0x50008), C.ERR_INVALID_ARG),
    (dict(K=0), C.ERR_UNSUPPORTED_SHAPE), (dict(K=33), C.ERR_UNSUPPORTED_SHAPE), (dict(H=12), C.ERR_UNSUPPORTED_SHAPE),
    (dict(H=0), C.ERR_UNSUPPORTED_SHAPE), (dict(M=-1), C.ERR_INVALID_ARG), (dict(n_rows=-1), C.ERR_INVALID_ARG),
    (dict(M=1 << 28), C.ERR_UNSUPPORTED_SHAPE), (dict(out=0x40010), C.ERR_INVALID_ARG),
])
def test_combine_arguments_refused(lib, kw, code):
    assert lib.clover_moe_combine(*dict(COMBINE, **kw).values()) == code
    assert C.last_error()


def test_combine_nothing_to_do(lib):
    assert lib.clover_moe_combine(*dict(COMBINE, M=0, y=None, pos=None, w=None, out=None).values()) == C.OK


def test_wrappers_refuse_host_tensors(lib):
    r = C.make_routing(8, 2)
    bad = [lambda: C.route(r, torch.zeros(4, 8)), lambda: C.quantize_fp4(torch.zeros(4, 64)),
           lambda: C.moe_combine(torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32),
                                 torch.zeros(2, 2))]
    q = C.Fp4(C.FP4_NV, torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))
    bad += [lambda: C.dequantize_fp4(q), lambda: C.fp4_product(q, q)]
    for f in bad:
        with pytest.raises(C.CloverError):
            f()


def test_fp4_parts_are_checked_and_kept(lib):
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    q = C.Fp4(C.FP4_NV, codes, scales)
    assert (q.mats, q.rows, q.cols, q.groups) == (1, 4, 64, 0)
    with pytest.raises(AttributeError):
        q.scales = scales[:1]
    with pytest.raises(AttributeError):
        q.codes = codes[:1]
    for off in (torch.zeros(3, dtype=torch.int32), torch.zeros(3), torch.zeros(1, 3, dtype=torch.int32)):
        with pytest.raises(C.CloverError):
            q.offsets = off  # two groups need two row tiles of scales; another type; another shape
    q.offsets = torch.zeros(2, dtype=torch.int32)
    assert q.groups == 1
    for bad in (lambda: C.Fp4(C.FP4_NV, codes, scales[:511]), lambda: C.Fp4(C.FP4_NV, codes.float(), scales),
                lambda: C.Fp4(C.FP4_NV, codes[:, ::2], scales), lambda: C.Fp4(2, codes, scales),
                lambda: C.Fp4(C.FP4_NV, codes[None], scales, offsets=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(C.CloverError):
            bad()


def test_counts_past_32_bits_refused():
    for kw in (dict(n_experts=(1 << 32) + 8, top_k=2), dict(n_experts=8, top_k=(1 << 32) + 2),
               dict(n_experts=8, top_k=2, n_groups=1 << 40)):
        with pytest.raises(C.CloverError):
            C.make_routing(**kw)


# ----------------------------------------------------------------- oracle pins


def test_e4m3_and_e2m1_tables():
    f8 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.E4M3, f8)
    assert np.isnan(R.e4m3_value(0x7F)) and R.e4m3_value(0x80 | 0x38) == -1.0
    # ties go to the even code, everything past 6 to 6
    for v, want in ((0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (0.26, 1), (4.9, 6), (1e9, 7)):
        assert R.nearest(R.E2M1, v) == want, v


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_oracle_round_trip(fmt):
    """Values that the format holds come back; a block's error is at most half of the widest step below its maximum."""
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, size=(5, 64)).astype(np.uint8)
    codes[:, ::16] = 7  # every block's largest value is 6
    if fmt == "nv":
        sb = rng.integers(40, 80, size=(5, 4)).astype(np.uint8)
    else:
        sb = rng.integers(100, 140, size=(5, 2)).astype(np.uint8)
    x = R.dequantize(codes, sb, fmt)
    c2, s2 = R.quantize(x, fmt)
    assert np.array_equal(s2, sb) and np.array_equal(c2, codes)
    x = rng.normal(size=(4, 128)).astype(np.float32)
    d = R.dequantize(*R.quantize(x, fmt), fmt)
    block = 16 if fmt == "nv" else 32
    amax = np.abs(x).reshape(4, -1, block).max(-1).repeat(block, 1).reshape(4, 128)
    # widest step 2 (between 4 and 6) times the scale: NV s <= amax / 6 * (1 + 1/16), saturation costs amax - 6 s <=
    # amax / 17; MX s <= amax / 4, saturation costs less than 2 s
    assert np.all(np.abs(d - x) <= (amax / 6 * 17 / 16 if fmt == "nv" else amax / 2))


def test_oracle_scale_places_are_a_permutation():
    seen = {R.scale_place(r, b) for r in range(256) for b in range(8)}
    assert len(seen) == 256 * 8
    assert R.scale_place(33, 2) == (0, 0, 16 + 4 + 2)
    off = [0, 0, 130, 131, 131, 400]
    rows = [R.grouped_scale_row(i, off) for i in range(400)]
    assert len(set(rows)) == 400 and max(rows) < (400 // 128 + 5) * 128


def test_oracle_route_by_hand():
    z = np.array([[0.0, 2.0, 1.0, -np.inf], [-np.inf] * 4, [np.nan, 1.0, 1.0, 0.0]])
    r = R.route(z, 2)
    assert r["idx"].tolist() == [[1, 2], [-1, -1], [1, 2]]
    e = np.exp(-1.0)
    assert np.allclose(r["w"][0], [1 / (1 + e), e / (1 + e)]) and r["w"][1].tolist() == [0, 0]
    assert r["offsets"].tolist() == [0, 0, 2, 4, 4] and r["rows"].tolist() == [0, 4, 1, 5]
    assert r["pos"].tolist() == [[0, 2], [-1, -1], [1, 3]]
    # the bias moves the choice, not the weight; groups of two, one kept by its two best
    z = np.array([[3.0, -3.0, 1.0, 1.0]])
    r = R.route(z, 1, score="sigmoid", bias=np.array([0, 0, 0, 1.0]), renormalise=False, scale=2.0)
    assert r["idx"].tolist() == [[3]] and np.allclose(r["w"], 2 / (1 + np.exp(-1.0)))
    r = R.route(z, 2, score="sigmoid", n_groups=2, top_groups=1, group_rank=2)
    assert r["idx"].tolist() == [[2, 3]]
    r = R.route(z, 2, score="sigmoid", n_groups=2, top_groups=1, group_rank=1)
    assert r["idx"].tolist() == [[0, 1]]


PRODUCT = dict(fmt=0, a=0x10000, sa=0x20000, n_rows=10, b=0x30000, sb=0x40000, offsets=0x50000, groups=4, N=64, K=256,
               alpha=1.0, group_alpha=None, epilogue=0, y=0x60000, ws=0x100000, nbytes=256, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), C.ERR_INVALID_ARG), (dict(K=96), C.ERR_UNSUPPORTED_SHAPE), (dict(K=0), C.ERR_UNSUPPORTED_SHAPE),
    (dict(N=0), C.ERR_UNSUPPORTED_SHAPE), (dict(N=63, epilogue=1), C.ERR_UNSUPPORTED_SHAPE),
    (dict(N=(1 << 24) + 1), C.ERR_UNSUPPORTED_SHAPE), (dict(epilogue=2), C.ERR_INVALID_ARG),
    (dict(groups=0), C.ERR_UNSUPPORTED_SHAPE), (dict(groups=513), C.ERR_UNSUPPORTED_SHAPE),
    (dict(n_rows=-1), C.ERR_UNSUPPORTED_SHAPE), (dict(n_rows=(1 << 29) + 1), C.ERR_UNSUPPORTED_SHAPE),
    (dict(offsets=None), C.ERR_INVALID_ARG), (dict(offsets=0x50002), C.ERR_INVALID_ARG),
    (dict(a=None), C.ERR_INVALID_ARG), (dict(sa=0x20008), C.ERR_INVALID_ARG), (dict(b=0x30004), C.ERR_INVALID_ARG),
    (dict(sb=None), C.ERR_INVALID_ARG), (dict(y=None), C.ERR_INVALID_ARG), (dict(y=0x60008), C.ERR_INVALID_ARG),
    (dict(group_alpha=0x70001), C.ERR_INVALID_ARG), (dict(ws=None), C.ERR_INVALID_ARG),
    (dict(ws=0x100010), C.ERR_INVALID_ARG), (dict(nbytes=255), C.ERR_WORKSPACE_TOO_SMALL),
    (dict(alpha=float("inf")), C.ERR_INVALID_ARG), (dict(alpha=float("nan")), C.ERR_INVALID_ARG),
])
def test_product_arguments_refused(lib, kw, code):
    assert lib.clover_fp4_product(*dict(PRODUCT, **kw).values()) == code
    assert C.last_error()


def test_product_nothing_to_do(lib):
    assert lib.clover_fp4_product_workspace_bytes() == 256
    assert lib.clover_fp4_product(*dict(PRODUCT, n_rows=0, a=None, b=None, y=None).values()) == C.OK


PLAN = r"""
#include <cstdio>
#include "plan.h"
using namespace clover::plan;
int main() {
  const int pairs[][4] = {{1024, 1, 8192, 0}, {1023, 1, 8192, 0}, {3402, 3, 8192, 0}, {1150, 1, 4096, 1}, {4132, 4, 4288, 1},
                          {3075, 3, 4160, 1}, {8192, 1, 4096, 0}, {65536, 256, 8192, 1}};
  for (auto& p : pairs) printf("pair %d\n", fp4_pairs(p[0], p[1], p[2], p[3] != 0) ? 1 : 0);
  for (int t = 1; t <= 200000; t += t < 2000 ? 1 : 997) {
    const RouteShape s = route_shape(t);
    printf("%d %d %d %d %d\n", t, s.cta_tokens, s.ctas, s.cluster ? 1 : 0, route_max_ctas(t));
  }
  return 0;
}
"""


def test_route_shapes(tmp_path):
    """Every token has a place, a CTA's tokens fit its 64-bit masks, a cluster is of at
    most 8 CTAs, a workspace holds every launch."""
    import os
    import shutil
    import subprocess
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    (tmp_path / "p.cpp").write_text(PLAN)
    subprocess.run([cxx, "-std=c++17", "-I", B.CSRC, str(tmp_path / "p.cpp"), "-o", str(tmp_path / "p")], check=True)
    out = subprocess.run([str(tmp_path / "p")], check=True, capture_output=True, text=True, cwd=os.fspath(tmp_path)).stdout
    # the product's rule, at the shapes the tests of its two forms use
    lines = out.splitlines()
    assert [x.split()[1] for x in lines if x.startswith("pair")] == ["1", "0", "1", "1", "1", "1", "0", "0"]
    held = 0
    for line in [x for x in lines if not x.startswith("pair")]:
        tokens, per, ctas, cluster, most = map(int, line.split())
        assert per * ctas >= tokens and per <= 64, line
        assert ctas in (1, 2, 4, 8) if cluster else (ctas - 1) * per < tokens, line
        # a workspace holds the counts of every call of its tokens or fewer
        assert cluster or ctas <= most, line
        assert most >= held, line
        held = most


def test_product_shared_workspace_arguments(lib):
    assert lib.clover_fp4_product_shared_workspace(None) == C.ERR_INVALID_ARG


def test_fp4_fields_cannot_be_set(lib):
    """Sizes and format are what the parts were checked for: another value would reach past them."""
    q = C.Fp4(C.FP4_MX, torch.zeros(2, 4, 32, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8))
    for name, value in dict(fmt=C.FP4_NV, device="cuda", mats=9, rows=400, cols=6400, groups=3).items():
        with pytest.raises(AttributeError):
            setattr(q, name, value)
    assert (q.fmt, q.device, q.mats, q.rows, q.cols, q.groups) == (C.FP4_MX, torch.device("cpu"), 2, 4, 64, 0)
    q.scale_exp = 3


def test_sizes_past_32_bits_refused(lib):
    """A count that would wrap on its way to the library is refused, not taken for the wrapped one."""
    big = (1 << 32) + 1
    r = C.make_routing(8, 2)
    codes = torch.zeros(1, 1, dtype=torch.uint8).expand(big, 32)  # (never contiguous, so only its shape counts)
    for f in (lambda: C.route_workspace_bytes(r, big), lambda: C.fp4_scale_bytes(C.FP4_NV, 1, big, 64),
              lambda: C.fp4_scale_bytes(C.FP4_NV, big, 1, 64), lambda: C.fp4_scale_bytes(C.FP4_NV, 1, 1, (1 << 32) + 64),
              lambda: C.fp4_scale_bytes(C.FP4_NV, 1, 1, 64, big), lambda: C.fp4_scale_bytes(1 << 32, 1, 1, 64),
              lambda: C.Fp4(C.FP4_NV, codes, torch.zeros(512, dtype=torch.uint8)),
              lambda: C.Fp4(1 << 32, torch.zeros(1, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))):
        with pytest.raises(C.CloverError):
            f()
    assert C.fp4_scale_bytes(C.FP4_NV, 1, 1, 64) == 512


def test_malformed_arguments_are_refused(lib, monkeypatch):
    """What the checks once met with an IndexError, KeyError or OverflowError of their own."""
    monkeypatch.setattr(C, "_on_current", lambda name, t: -1)  # (host tensors: every call here is refused before the library's)
    monkeypatch.setattr(C, "_current_stream", lambda dev: None)
    r = C.make_routing(8, 2)
    z, x, i32 = torch.zeros(4, 8), torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)
    some = {"idx": torch.zeros(4, 2, dtype=torch.int32), "w": torch.zeros(4, 2)}
    ws = torch.zeros(4096, dtype=torch.uint8)
    q = C.Fp4(C.FP4_NV, torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), scale_exp=4000)
    for f in (lambda: C.quantize_fp4(x, offsets=i32[0]), lambda: C.quantize_fp4(x, offsets=i32, src_rows=i32[0]),
              lambda: C.route(r, z, ws=ws, out=some), lambda: C.route(r, z, ws=ws, out={}, grouping=False),
              lambda: C.fp4_product(q, q, ws=ws)):
        with pytest.raises(C.CloverError):
            f()


# --------------------------------------------------- streams of the binding


class _Calls:
    """Stands in for the library: every launch succeeds, its stream is kept, sizes are ordinary."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def f(*args):
            if name.endswith("_bytes"):
                return 4096
            if not name.endswith("_shared_workspace"):
                self.streams.append(args[-1].value if isinstance(args[-1], ctypes.c_void_p) else args[-1])
            return C.OK
        return f


def _calls_with_streams():
    from block_diffusion_moe_gb300 import synth
    d = synth.TINY
    x, z, y = torch.zeros(4, 64), torch.zeros(4, 8), torch.zeros(8, 64, dtype=torch.bfloat16)
    pos, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    q = C.Fp4(C.FP4_NV, torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4096, dtype=torch.uint8))
    r = C.make_routing(8, 2)
    return [lambda s: C.route(r, z, stream=s), lambda s: C.quantize_fp4(x, stream=s), lambda s: C.dequantize_fp4(q, stream=s),
            lambda s: C.fp4_product(q, q, stream=s), lambda s: C.moe_combine(y, pos, w, stream=s),
            lambda s: C.lmhead_unmask(d, y, torch.zeros(4, d.hidden), pos, pos, stream=s),
            lambda s: C.lmhead_accept(d, y, torch.zeros(4, d.hidden), pos, 2, stream=s)]


def test_calls_allocate_on_their_stream(monkeypatch):
    """What a call with stream= makes (workspaces, results) is made while that stream is current, and the launch goes to
    it: a block made under another stream is filled, reused and freed in that one's order."""
    import contextlib
    import types
    fake = _Calls()
    current, made = [111], []

    @contextlib.contextmanager
    def as_current(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    def spy(f):
        def g(*a, **kw):
            made.append(current[-1])
            return f(*a, **kw)
        return g

    side = types.SimpleNamespace(cuda_stream=222, device=torch.device("cpu"))
    calls = _calls_with_streams()
    monkeypatch.setattr(C, "lib", lambda: fake)
    monkeypatch.setattr(C, "_on_current", lambda name, t: -1)  # (host tensors stand in for the device's)
    monkeypatch.setattr(C, "_current_stream", lambda dev: current[-1])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=current[-1]))
    monkeypatch.setattr(torch.cuda, "stream", as_current)
    monkeypatch.setattr(torch, "empty", spy(torch.empty))
    monkeypatch.setattr(torch, "zeros", spy(torch.zeros))
    for i, f in enumerate(calls):
        for s, want in ((side, 222), (None, 111)):
            made.clear()
            fake.streams.clear()
            f(s)
            assert fake.streams == [want], (i, fake.streams)
            if i != 5 and i != 6:
                assert made and all(m == want for m in made), (i, made)
            else:  # (the call's own inputs are made before it)
                assert all(m == want for m in made[1:]), (i, made)
        assert current == [111]


def test_streams_of_another_device_refused():
    import types
    other = types.SimpleNamespace(cuda_stream=222, device=torch.device("cuda", 1))
    B.build()
    for f in _calls_with_streams():
        with pytest.raises(C.CloverError):
            f(other)
