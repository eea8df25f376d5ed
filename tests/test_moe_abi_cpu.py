"""Host-side checks of the mixture-of-experts entry points (no GPU needed): every function of
include/fp8blk_moe.h is exported, bad arguments get the documented status before any device work, and the binding
refuses tensors that the library could not check."""

import ctypes
import os
import re

import pytest
import torch

import block_scaled_fp8_amax_amd as fb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8blk_moe.h")
OK, INVALID, SHAPE, ALIGN, UNSUP = 0, 1, 2, 3, 4
P = 0x10000          # a fake, aligned address (never dereferenced)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return fb.library()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(fp8_\w+)\s*\(", text, flags=re.M))
    assert names == {n for n in fb.moe.__all__ if n.startswith("fp8_")}
    raw = ctypes.CDLL(fb.library_path)
    assert all(hasattr(raw, n) for n in names)
    assert lib.fp8_moe_abi_version() == 1


def _caller(fn, names, values):
    def call(**kw):
        a = dict(zip(names, values))
        assert not set(kw) - set(a), kw
        a.update(kw)
        return fn(*[a[n] for n in names], None)
    return call


def test_rmsnorm_quantize_validation(lib):
    call = _caller(lib.fp8_rmsnorm_quantize,
                   "x res w wt rows cols eps kind rule q scale h y ydq rstd".split(),
                   [P, P, P, 1, 4, 256, 1e-6, 1, 0, P, P, P, P, P, P])
    assert call(kind=2) == UNSUP and call(kind=3) == INVALID
    assert call(kind=0, rule=2) == INVALID and call(wt=2) == INVALID
    for eps in (0.0, -1.0, 1e-21, NAN, INF):
        assert call(eps=eps) == INVALID, eps
    assert call(h=None) == INVALID and call(res=None) == INVALID          # h and residual go together
    assert call(cols=192) == SHAPE and call(kind=0, cols=48) == SHAPE
    assert call(cols=32768 + 128) == SHAPE and call(rows=-1) == SHAPE and call(rows=1 << 31) == SHAPE
    assert call(x=None) == INVALID and call(w=None) == INVALID and call(q=None) == INVALID
    assert call(scale=None) == INVALID
    for name in "x res w q h y ydq".split():
        assert call(**{name: P + 8}) == ALIGN, name
    assert call(scale=P + 2) == ALIGN and call(rstd=P + 2) == ALIGN
    assert call(rows=0, x=None, w=None, q=None, scale=None) == OK and call(cols=0) == OK


def test_rmsnorm_backward_validation(lib):
    size = ctypes.c_size_t(0)
    need = lib.fp8_rmsnorm_backward_workspace
    assert need(4, 256, None) == INVALID and need(-1, 256, ctypes.byref(size)) == SHAPE
    assert need(4, 252, ctypes.byref(size)) == SHAPE and need(4, 32776, ctypes.byref(size)) == SHAPE
    assert need(0, 256, ctypes.byref(size)) == OK and size.value == 0
    assert need(4, 256, ctypes.byref(size)) == OK and size.value >= 256 * 4
    call = _caller(lib.fp8_rmsnorm_backward, "dy h w wt rstd dres rows cols ws bytes dx dw".split(),
                   [P, P, P, 1, P, P, 4, 256, P, size.value, P, P])
    assert call(wt=2) == INVALID and call(bytes=size.value - 1) == INVALID and call(ws=None) == INVALID
    for name in "dy h w rstd dx dw".split():
        assert call(**{name: None}) == INVALID, name
    for name in "dy h w dres dx".split():
        assert call(**{name: P + 8}) == ALIGN, name
    assert call(ws=P + 128) == ALIGN and call(rstd=P + 1) == ALIGN and call(dw=P + 2) == ALIGN
    assert call(cols=260) == SHAPE and call(rows=-4) == SHAPE and call(cols=0) == OK


def test_route_validation(lib):
    names = "logits lt bias tokens experts k score groups kept gs renorm scale ids w".split()
    call = _caller(lib.fp8_moe_route, names, [P, 1, P, 4, 64, 8, 1, 8, 4, 1, 1, 1.0, P, P])
    assert call(lt=2) == INVALID and call(score=2) == INVALID and call(gs=2) == INVALID and call(renorm=2) == INVALID
    assert call(scale=NAN) == INVALID and call(scale=INF) == INVALID
    assert call(experts=0) == INVALID and call(experts=1025, groups=1, kept=1) == INVALID
    assert call(k=0) == INVALID and call(k=65) == INVALID
    assert call(groups=0) == INVALID and call(groups=65) == INVALID and call(groups=7) == INVALID
    assert call(kept=0) == INVALID and call(kept=9) == INVALID
    assert call(k=33, kept=4) == INVALID                                  # more than the kept groups hold
    assert call(tokens=-1) == SHAPE and call(tokens=1 << 28) == SHAPE
    assert call(logits=None) == INVALID and call(ids=None) == INVALID and call(w=None) == INVALID
    assert call(logits=P + 2) == ALIGN and call(lt=0, logits=P + 1) == ALIGN and call(bias=P + 2) == ALIGN
    assert call(ids=P + 2) == ALIGN and call(w=P + 1) == ALIGN
    assert call(tokens=0, logits=None, ids=None, w=None) == OK
    back = _caller(lib.fp8_moe_route_backward, "logits lt ids dw tokens experts k score renorm scale dl".split(),
                   [P, 1, P, P, 4, 64, 8, 1, 1, 1.0, P])
    assert back(lt=3) == INVALID and back(score=-1) == INVALID and back(renorm=-1) == INVALID
    assert back(scale=NAN) == INVALID and back(experts=0) == INVALID and back(k=65) == INVALID
    assert back(tokens=-1) == SHAPE and back(tokens=0) == OK
    for name in "logits ids dw dl".split():
        assert back(**{name: None}) == INVALID and back(**{name: P + 2}) == ALIGN, name


def test_plan_validation(lib):
    size = ctypes.c_size_t(7)
    need = lib.fp8_moe_plan_workspace
    assert need(8, 8, 64, None) == INVALID and need(-1, 8, 64, ctypes.byref(size)) == SHAPE
    assert need(8, 0, 64, ctypes.byref(size)) == INVALID and need(8, 8, 1025, ctypes.byref(size)) == INVALID
    assert need(8, 8, 64, ctypes.byref(size)) == OK and size.value == 0
    assert need(1 << 14, 8, 256, ctypes.byref(size)) == OK and 0 < size.value <= 1 << 20
    big = size.value
    # a count per expert and 2048 pairs
    assert need(1 << 24, 64, 1024, ctypes.byref(size)) == OK and size.value == ((1 << 19) + 1) * 1024 * 4
    assert need((1 << 24) + 1, 64, 1024, ctypes.byref(size)) == SHAPE
    call = _caller(lib.fp8_moe_plan, "ids tokens k experts ws bytes off row slot".split(),
                   [P, 1 << 14, 8, 256, P, big, P, P, P])
    assert call(ws=None) == INVALID and call(bytes=big - 1) == INVALID and call(ws=P + 8) == ALIGN
    for name in "ids off row slot".split():
        assert call(**{name: None}) == INVALID and call(**{name: P + 2}) == ALIGN, name
    assert call(experts=0) == INVALID and call(k=65) == INVALID and call(tokens=-1) == SHAPE


def test_matvec_validation(lib):
    call = _caller(lib.fp8_nvfp4_matvec, "x q bs gs rpt m n k y yt".split(), [P, P, P, P, 64, 1, 128, 256, P, 0])
    assert call(yt=2) == INVALID
    assert call(k=0) == SHAPE and call(k=24) == SHAPE and call(k=(1 << 24) + 16) == SHAPE
    assert call(m=-1) == SHAPE and call(m=1 << 31) == SHAPE and call(n=-1) == SHAPE and call(n=(1 << 24) + 64) == SHAPE
    assert call(rpt=0) == SHAPE and call(rpt=48) == SHAPE
    for name in "x q bs gs y".split():
        assert call(**{name: None}) == INVALID, name
    assert call(x=P + 8) == ALIGN and call(q=P + 4) == ALIGN and call(gs=P + 2) == ALIGN
    assert call(y=P + 1) == ALIGN and call(yt=1, y=P + 2) == ALIGN
    assert call(m=0, x=None) == OK and call(n=0, q=None) == OK
    grp = _caller(lib.fp8_nvfp4_grouped_matvec, "x xr ri q bs gs rpt off groups m n k y yt".split(),
                  [P, 4, P, P, P, P, 128, P, 8, 16, 128, 256, P, 0])
    assert grp(groups=0) == INVALID and grp(groups=1025) == INVALID and grp(yt=-1) == INVALID
    assert grp(xr=-1) == SHAPE and grp(xr=0) == SHAPE and grp(ri=None) == SHAPE      # x[i] needs as many rows
    assert grp(rpt=100) == SHAPE and grp(k=8) == SHAPE
    for name in "x q bs gs off y".split():
        assert grp(**{name: None}) == INVALID, name
    assert grp(off=P + 2) == ALIGN and grp(ri=P + 2) == ALIGN and grp(x=P + 2) == ALIGN
    assert grp(m=0, x=None, xr=0) == OK


def test_combine_validation(lib):
    call = _caller(lib.fp8_moe_combine, "rows rt total slot w res tokens k n y yt".split(),
                   [P, 0, 32, P, P, P, 4, 8, 128, P, 0])
    back = _caller(lib.fp8_moe_combine_backward, "dy dt rows rt total slot w tokens k n dr dw".split(),
                   [P, 0, P, 0, 32, P, P, 4, 8, 128, P, P])
    assert call(rt=2) == INVALID and call(yt=2) == INVALID and back(rt=2) == INVALID and back(dt=2) == INVALID
    for f in (call, back):
        assert f(k=0) == INVALID and f(k=65) == INVALID
        assert f(n=4) == SHAPE and f(n=-8) == SHAPE and f(n=(1 << 24) + 8) == SHAPE
        assert f(tokens=-1) == SHAPE and f(total=-1) == SHAPE and f(total=1 << 31) == SHAPE
        assert f(rows=None) == INVALID and f(slot=None) == INVALID and f(w=None) == INVALID
        assert f(rows=P + 8) == ALIGN and f(slot=P + 2) == ALIGN and f(w=P + 2) == ALIGN
        assert f(tokens=0) == OK
    assert call(y=None) == INVALID and call(y=P + 4) == ALIGN and call(res=P + 8) == ALIGN and call(n=0) == OK
    assert back(dy=None) == INVALID and back(dr=None) == INVALID and back(dw=None) == INVALID
    assert back(dy=P + 8) == ALIGN and back(dr=P + 8) == ALIGN and back(dw=P + 2) == ALIGN


# ------------------------------------------------------------------- binding

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_host_tensors(lib):
    with pytest.raises(ValueError, match="on a GPU"):
        fb.rmsnorm_quantize(z(2, 128), z(128), 1e-6)
    with pytest.raises(ValueError, match="on a GPU"):
        fb.rmsnorm_backward(z(2, 128), z(2, 128), z(128), z(2, dtype=F32))
    with pytest.raises(ValueError, match="on a GPU"):
        fb.moe_route(z(2, 8), 2)
    with pytest.raises(ValueError, match="on a GPU"):
        fb.moe_route_backward(z(2, 8), z(2, 2, dtype=I32), z(2, 2, dtype=F32))
    with pytest.raises(ValueError, match="on a GPU"):
        fb.moe_plan(z(2, 2, dtype=I32), 8)
    with pytest.raises(ValueError, match="on a GPU"):
        fb.nvfp4_matvec(z(2, 32), z(4, 16, dtype=U8), z(4, 2, dtype=U8), z(1, dtype=F32))
    with pytest.raises(ValueError, match="on a GPU"):
        fb.nvfp4_grouped_matvec(z(2, 32), z(3, 4, 16, dtype=U8), z(3, 4, 2, dtype=U8), z(3, dtype=F32),
                                z(4, dtype=I32))
    with pytest.raises(ValueError, match="on a GPU"):
        fb.moe_combine(z(4, 8), z(2, 2, dtype=I32), z(2, 2, dtype=F32))
    with pytest.raises(ValueError, match="on a GPU"):
        fb.moe_combine_backward(z(2, 8), z(4, 8), z(2, 2, dtype=I32), z(2, 2, dtype=F32))


def test_binding_checks_types_shapes_and_strides(lib):
    def norm(**kw):
        a = {"x": z(4, 256), "w": z(256), "q": z(4, 256, dtype=U8), "scale": z(4, 2, dtype=F32), "kind": "1x128",
             "rule": "ceil"}
        more = {k: kw.pop(k) for k in list(kw) if k not in a}
        a.update(kw)
        fb.fp8_rmsnorm_quantize(a["x"], a["w"], 1e-6, a["kind"], a["rule"], a["q"], a["scale"], **more)

    for bad, text in (({"x": z(4, 256, dtype=torch.float16)}, "x has dtype"), ({"x": z(256)}, "x must have 2"),
                      ({"x": None}, "x must be a tensor"), ({"w": z(128)}, "weight has shape"),
                      ({"w": z(256, dtype=torch.float64)}, "weight has dtype"), ({"q": z(4, 256)}, "q has dtype"),
                      ({"scale": z(2, 4, dtype=F32)}, "scale has shape"), ({"kind": "1x32"}, "scale has dtype"),
                      ({"kind": "128x128"}, "kind '128x128'"), ({"rule": "round"}, "rule 'round'"),
                      ({"x": z(256, 4).t()}, "x must be contiguous"), ({"y": z(4, 128)}, "y has shape"),
                      ({"residual": z(4, 256), "h": z(4, 256, dtype=F32)}, "h has dtype"),
                      ({"rstd": z(5, dtype=F32)}, "rstd has shape")):
        with pytest.raises(ValueError, match=text):
            norm(**bad)
    with pytest.raises(ValueError, match="dweight has dtype"):
        fb.fp8_rmsnorm_backward(z(2, 64), z(2, 64), z(64), z(2, dtype=F32), z(4096, dtype=U8), z(2, 64),
                                z(64, dtype=F32))
    with pytest.raises(ValueError, match="ids has shape"):
        fb.fp8_moe_route(z(2, 8), z(3, 2, dtype=I32), z(3, 2, dtype=F32))
    with pytest.raises(ValueError, match="ids has dtype"):
        fb.fp8_moe_route(z(2, 8), z(2, 2, dtype=torch.int64), z(2, 2, dtype=F32))
    with pytest.raises(ValueError, match="score 'relu'"):
        fb.fp8_moe_route(z(2, 8), z(2, 2, dtype=I32), z(2, 2, dtype=F32), score="relu")
    with pytest.raises(ValueError, match="bias has shape"):
        fb.fp8_moe_route(z(2, 8), z(2, 2, dtype=I32), z(2, 2, dtype=F32), bias=z(4, dtype=F32))
    with pytest.raises(ValueError, match="dlogits has dtype"):
        fb.fp8_moe_route_backward(z(2, 8), z(2, 2, dtype=I32), z(2, 2, dtype=F32), z(2, 8, dtype=F32))
    with pytest.raises(ValueError, match="offsets has shape"):
        fb.fp8_moe_plan(z(2, 2, dtype=I32), 8, None, z(8, dtype=I32), z(4, dtype=I32), z(2, 2, dtype=I32))
    with pytest.raises(ValueError, match="slot must be contiguous"):
        fb.fp8_moe_plan(z(2, 2, dtype=I32), 8, None, z(9, dtype=I32), z(4, dtype=I32), z(2, 2, dtype=I32).t())
    with pytest.raises(ValueError, match="block_scale has shape"):
        fb.nvfp4_matvec(z(2, 32), z(4, 16, dtype=U8), z(4, 1, dtype=U8), z(1, dtype=F32))
    with pytest.raises(ValueError, match="q has shape"):
        fb.nvfp4_matvec(z(2, 64), z(4, 16, dtype=U8), z(4, 4, dtype=U8), z(1, dtype=F32))
    with pytest.raises(ValueError, match="does not divide"):
        fb.nvfp4_matvec(z(2, 32), z(4, 16, dtype=U8), z(4, 2, dtype=U8), z(1, dtype=F32), rows_per_tensor=3)
    with pytest.raises(ValueError, match="must agree"):
        fb.fp8_nvfp4_grouped_matvec(z(2, 32), None, z(3, 4, 16, dtype=U8), z(3, 4, 2, dtype=U8), z(3, dtype=F32), 4,
                                    z(4, dtype=I32), z(5, 4))
    with pytest.raises(ValueError, match="group_offsets has shape"):
        fb.nvfp4_grouped_matvec(z(2, 32), z(3, 4, 16, dtype=U8), z(3, 4, 2, dtype=U8), z(3, dtype=F32),
                                z(3, dtype=I32))
    with pytest.raises(ValueError, match="weights has shape"):
        fb.moe_combine(z(4, 8), z(2, 2, dtype=I32), z(2, 3, dtype=F32))
    with pytest.raises(ValueError, match="drows has dtype"):
        fb.fp8_moe_combine_backward(z(2, 8), z(4, 8), z(2, 2, dtype=I32), z(2, 2, dtype=F32), z(4, 8, dtype=F32),
                                    z(2, 2, dtype=F32))
