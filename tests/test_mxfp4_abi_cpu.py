"""Host-side checks of the MXFP4 experts' entry points (no GPU needed): every function of include/fp8blk_mxfp4.h is
exported, bad arguments get the documented status before any device work, and the binding refuses tensors that the
library could not check."""

import ctypes
import os
import re

import pytest
import torch

import block_scaled_fp8_amax_amd as fb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8blk_mxfp4.h")
OK, INVALID, SHAPE, ALIGN, UNSUP = 0, 1, 2, 3, 4
P = 0x10000          # a fake, aligned address (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    return fb.library()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(fp8_\w+)\s*\(", text, flags=re.M))
    assert names == {n for n in fb.mxfp4.__all__ if n.startswith("fp8_")}
    raw = ctypes.CDLL(fb.library_path)
    assert all(hasattr(raw, n) for n in names)
    assert lib.fp8_mxfp4_abi_version() == 1


def _caller(fn, names, values):
    def call(**kw):
        a = dict(zip(names, values))
        assert not set(kw) - set(a), kw
        a.update(kw)
        return fn(*[a[n] for n in names], None)
    return call


def test_codec_validation(lib):
    call = _caller(lib.fp8_mxfp4_quantize, "x rows cols rule q scale xdq".split(), [P, 4, 64, 0, P, P, P])
    assert call(rule=2) == INVALID and call(rule=-1) == INVALID
    assert call(cols=48) == SHAPE and call(cols=-32) == SHAPE and call(rows=-1) == SHAPE
    assert call(rows=1 << 28, cols=1 << 10) == SHAPE
    for name in "x q scale".split():
        assert call(**{name: None}) == INVALID, name
    for name in "x q xdq".split():
        assert call(**{name: P + 8}) == ALIGN, name
    assert call(rows=0, x=None) == OK and call(cols=0, q=None) == OK
    back = _caller(lib.fp8_mxfp4_dequantize, "q scale rows cols x".split(), [P, P, 4, 64, P])
    assert back(cols=16) == SHAPE and back(rows=-1) == SHAPE and back(rows=1 << 28, cols=1 << 10) == SHAPE
    for name in "x q scale".split():
        assert back(**{name: None}) == INVALID, name
    assert back(q=P + 8) == ALIGN and back(x=P + 2) == ALIGN and back(rows=0, q=None) == OK


def test_product_validation(lib):
    call = _caller(lib.fp8_mxfp4_gemm, "a as_ elem b bs m n k y yt".split(), [P, P, 1, P, P, 4, 64, 256, P, 0])
    grouped = _caller(lib.fp8_mxfp4_grouped_gemm, "a as_ elem rows index b bs off groups m n k y yt".split(),
                      [P, P, 0, 9, P, P, P, P, 2, 4, 64, 256, P, 1])
    for c in (call, grouped):
        assert c(elem=2) == INVALID and c(elem=-1) == INVALID and c(yt=2) == INVALID
        assert c(k=64) == SHAPE and c(k=0) == SHAPE and c(k=(1 << 24) + 128) == SHAPE
        assert c(m=-1) == SHAPE and c(m=1 << 31) == SHAPE and c(n=-1) == SHAPE and c(n=(1 << 24) + 1) == SHAPE
        for name in "a as_ b bs y".split():
            assert c(**{name: None}) == INVALID, name
        for name in "a b y".split():
            assert c(**{name: P + 8}) == ALIGN, name
        assert c(as_=P + 2) == ALIGN and c(bs=P + 1) == ALIGN
        assert c(m=0, a=None) == OK and c(n=0, b=None) == OK
    assert grouped(groups=0) == INVALID and grouped(groups=1025) == INVALID and grouped(off=None) == INVALID
    assert grouped(off=P + 2) == ALIGN and grouped(index=P + 1) == ALIGN
    assert grouped(rows=0) == SHAPE and grouped(index=None) == SHAPE and grouped(rows=1 << 24) == SHAPE


def test_matvec_validation(lib):
    call = _caller(lib.fp8_mxfp4_matvec, "x q s m n k y yt".split(), [P, P, P, 4, 64, 96, P, 0])
    grouped = _caller(lib.fp8_mxfp4_grouped_matvec, "x rows index q s off groups m n k y yt".split(),
                      [P, 9, P, P, P, P, 2, 4, 64, 96, P, 1])
    for c in (call, grouped):
        assert c(yt=2) == INVALID and c(k=80) == SHAPE and c(k=0) == SHAPE and c(k=(1 << 24) + 32) == SHAPE
        assert c(m=-1) == SHAPE and c(n=-1) == SHAPE and c(n=(1 << 24) + 1) == SHAPE
        for name in "x q s y".split():
            assert c(**{name: None}) == INVALID, name
        assert c(x=P + 8) == ALIGN and c(q=P + 8) == ALIGN and c(y=P + 1) == ALIGN
        assert c(m=0, x=None) == OK and c(n=0, q=None) == OK
    assert call(yt=1, y=P + 2) == ALIGN
    assert call(m=1 << 20, k=1024) == SHAPE and grouped(rows=1 << 20, k=1024) == SHAPE
    assert grouped(groups=0) == INVALID and grouped(groups=1025) == INVALID and grouped(off=None) == INVALID
    assert grouped(rows=0) == SHAPE and grouped(index=None) == SHAPE and grouped(off=P + 1) == ALIGN
    assert grouped(index=P + 2) == ALIGN


def test_gradient_validation(lib):
    back = _caller(lib.fp8_grouped_dgrad, "dy w off groups m n k dx t".split(), [P, P, P, 2, 4, 64, 96, P, 0])
    wg = _caller(lib.fp8_grouped_wgrad, "dy x rows index off groups m n k dw t".split(),
                 [P, P, 9, P, P, 2, 4, 64, 96, P, 1])
    for c in (back, wg):
        assert c(t=2) == INVALID and c(groups=0) == INVALID and c(groups=1025) == INVALID
        assert c(n=60) == SHAPE and c(k=4) == SHAPE and c(n=-8) == SHAPE and c(m=-1) == SHAPE and c(m=1 << 31) == SHAPE
        assert c(n=1 << 16, k=1 << 15) == SHAPE and c(n=(1 << 22) + 8, k=8) == SHAPE and c(k=(1 << 22) + 8, n=8) == SHAPE
        assert c(dy=None) == INVALID and c(off=None) == INVALID and c(dy=P + 8) == ALIGN and c(off=P + 2) == ALIGN
        assert c(k=0, dy=None) == OK
    assert back(w=None) == INVALID and back(dx=None) == INVALID and back(w=P + 8) == ALIGN and back(dx=P + 8) == ALIGN
    assert back(m=0, dy=None) == OK
    assert wg(x=None) == INVALID and wg(dw=None) == INVALID and wg(x=P + 8) == ALIGN and wg(dw=P + 4) == ALIGN
    assert wg(rows=0) == SHAPE and wg(index=None) == SHAPE and wg(rows=1 << 25) == SHAPE and wg(index=P + 2) == ALIGN
    assert wg(n=0, dy=None) == OK


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_the_binding_refuses(lib):
    u8, i32, f32 = torch.uint8, torch.int32, torch.float32
    x, q, s = _t(4, 128), _t(4, 64, dtype=u8), _t(4, 4, dtype=u8)
    with pytest.raises(ValueError, match="GPU"):
        fb.fp8_mxfp4_quantize(x, "ceil", q, s)
    for bad in (dict(x=_t(4, 128, dtype=f32)), dict(q=_t(4, 128, dtype=u8)), dict(s=_t(4, 8, dtype=u8)),
                dict(x=_t(128, 4).t()), dict(rule="up"), dict(xdq=_t(4, 64)), dict(x=None), dict(x=_t(512))):
        a = dict(x=x, rule="ceil", q=q, s=s, xdq=None)
        a.update(bad)
        with pytest.raises(ValueError):
            fb.fp8_mxfp4_quantize(a["x"], a["rule"], a["q"], a["s"], a["xdq"])
    with pytest.raises(ValueError):
        fb.mxfp4_dequantize(q, _t(4, 2, dtype=u8))
    b, bs, y = _t(8, 64, dtype=u8), _t(8, 4, dtype=u8), _t(4, 8)
    for args in ((q, s, "e4m3", b, bs, y), (x, s, "e2m1", b, bs, y), (q, s, "e5m2", b, bs, y),
                 (q, s, "e2m1", b, bs, _t(8, 4)), (q, s, "e2m1", _t(8, 32, dtype=u8), bs, y),
                 (q, _t(4, 8, dtype=u8), "e2m1", b, bs, y), (q, s, "e2m1", b, bs, _t(4, 8, dtype=torch.float16))):
        with pytest.raises(ValueError):
            fb.fp8_mxfp4_gemm(*args)
    with pytest.raises(ValueError, match="GPU"):
        fb.fp8_mxfp4_gemm(q, s, "e2m1", b, bs, y)
    gb, gs, off = _t(3, 8, 64, dtype=u8), _t(3, 8, 4, dtype=u8), _t(4, dtype=i32)
    with pytest.raises(ValueError, match="agree"):
        fb.fp8_mxfp4_grouped_gemm(q, s, "e2m1", None, gb, gs, off, _t(5, 8))
    for idx, o in ((_t(5, dtype=torch.int64), off), (_t(4, dtype=i32), off), (_t(5, dtype=i32), _t(3, dtype=i32))):
        with pytest.raises(ValueError):
            fb.fp8_mxfp4_grouped_gemm(q, s, "e2m1", idx, gb, gs, o, _t(5, 8))
    with pytest.raises(ValueError, match="agree"):
        fb.fp8_mxfp4_grouped_matvec(x, None, gb, gs, off, _t(5, 8))
    with pytest.raises(ValueError):
        fb.fp8_mxfp4_matvec(x, b, bs, _t(4, 9))
    with pytest.raises(ValueError):
        fb.fp8_mxfp4_matvec(x.float(), b, bs, y)
    dy, w = _t(5, 8), _t(3, 8, 16)
    for args in ((dy, w, off, _t(5, 8)), (dy, _t(3, 16, 16), off, _t(5, 16)), (dy, w, _t(3, dtype=i32), _t(5, 16)),
                 (dy.float(), w, off, _t(5, 16)), (dy, w.transpose(1, 2), off, _t(5, 8))):
        with pytest.raises(ValueError):
            fb.fp8_grouped_dgrad(*args)
    with pytest.raises(ValueError, match="agree"):
        fb.fp8_grouped_wgrad(dy, _t(6, 16), None, off, _t(3, 8, 16))
    with pytest.raises(ValueError):
        fb.fp8_grouped_wgrad(dy, _t(6, 16), _t(6, dtype=i32), off, _t(3, 8, 16))
    with pytest.raises(ValueError, match="GPU"):
        fb.fp8_grouped_wgrad(dy, _t(5, 16), None, off, _t(3, 8, 16))
