"""GPU parity of fp8_mxfp4_gemm / fp8_mxfp4_grouped_gemm with float64 products of the decoded operands.

Two kinds of checks.  Values on a coarse binary grid make every product and every partial sum exact in fp32 whatever the
order of addition, so results are equal, bit for bit.  Random values: any order of k additions in fp32 is off by at most
k 2^-24 of the sum of magnitudes; E4M3 rows with bf16 results add 2^-10 of it (7 products of each run of 8 cut 13 bits
below the largest); a bf16 result 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import block_scaled_fp8_amax_amd as fb

pytestmark = pytest.mark.gpu
F64 = torch.float64
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=F64)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _scales(s):
    return torch.exp2(s.to(F64) - 127).repeat_interleave(32, -1)


def _matrix(q, s):
    t = E2M1.to(q.device)
    v = torch.stack([t[(q & 15).long()], t[(q >> 4).long()]], -1).flatten(-2)
    return v * _scales(s)


def _rows(a, s, elem):
    return _matrix(a, s) if elem == "e2m1" else a.view(torch.float8_e4m3fn).to(F64) * _scales(s)


def _bytes(g, *shape, lo=0, hi=256):
    return torch.randint(lo, hi, shape, device="cuda", generator=g, dtype=torch.int32).to(torch.uint8)


def _grid(g, m, n, k, elem, groups=None):
    """Any E2M1 codes, E4M3 codes of small integers, scales of 2^-1 .. 2^1."""
    b = _bytes(g, *(() if groups is None else (groups,)), n, k // 2)
    bs = _bytes(g, *b.shape[:-1], k // 32, lo=126, hi=129)
    if elem == "e2m1":
        a = _bytes(g, m, k // 2)
    else:
        a = (_bytes(g, m, k, hi=9).float() - 4).to(torch.float8_e4m3fn)
    return a, _bytes(g, m, k // 32, lo=126, hi=129), b, bs


def _random(g, m, n, k, elem, groups=None):
    """Quantized normal values, a few channels large, weights small."""
    x = torch.randn((m, k), device="cuda", generator=g)
    x[:, torch.randperm(k, device="cuda", generator=g)[: max(1, k // 100)]] *= 50
    x = x.to(torch.bfloat16)
    a, s = fb.mxfp4_quantize(x) if elem == "e2m1" else fb.quantize(x, "1x32")
    w = (0.02 * torch.randn(((groups or 1) * n, k), device="cuda", generator=g)).to(torch.bfloat16)
    b, bs = fb.mxfp4_quantize(w)
    if groups is not None:
        b, bs = b.view(groups, n, k // 2), bs.view(groups, n, k // 32)
    return a, s, b, bs


def _tolerance(want, mag, k, elem, dtype):
    tol = k * 2.0 ** -24 * mag
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
        if elem == "e4m3":
            tol = tol + 2.0 ** -10 * mag
    return tol


def _near(y, x, w, k, elem, dtype):
    want, mag = x @ w.T, x.abs() @ w.abs().T
    bad = ((y.to(F64) - want).abs() > _tolerance(want, mag, k, elem, dtype)).sum().item()
    assert bad == 0, f"{bad} of {y.numel()} results out of tolerance"


SHAPES = [(1, 1, 128), (1, 16, 256), (3, 100, 384), (16, 64, 512), (17, 33, 640), (33, 257, 128), (64, 128, 1024),
          (65, 130, 896), (100, 1000, 256), (128, 256, 1152), (129, 511, 512), (200, 48, 2048), (256, 512, 384),
          (300, 2002, 256), (513, 260, 768), (1000, 72, 512), (2, 4096, 7168), (40, 4100, 640)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_exact_on_a_grid(m, n, k, elem, dtype):
    print(f"[mx gemm] grid {m}x{n}x{k} {elem} {dtype}", flush=True)
    a, s, b, bs = _grid(_gen(m + n + k), m, n, k, elem)
    y = fb.mxfp4_gemm(a, s, elem, b, bs, out_dtype=dtype)
    want = (_rows(a, s, elem) @ _matrix(b, bs).T).to(dtype)
    assert torch.equal(y, want)


@pytest.mark.parametrize("m,n,k", [(5, 300, 7168), (130, 257, 1280), (600, 520, 512), (32, 96, 16384)])
@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_random(m, n, k, elem, dtype):
    print(f"[mx gemm] random {m}x{n}x{k} {elem} {dtype}", flush=True)
    a, s, b, bs = _random(_gen(m * n), m, n, k, elem)
    y = fb.mxfp4_gemm(a, s, elem, b, bs, out_dtype=dtype)
    _near(y, _rows(a, s, elem), _matrix(b, bs), k, elem, dtype)


@pytest.mark.parametrize("m,n", [(8, 40), (200, 300)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_e4m3_code(m, n, dtype):
    """All magnitudes side by side in a block: float results keep fp32 sums, bf16 ones the documented cut."""
    g = _gen(7)
    k = 512
    a = _bytes(g, m, k)
    a[(a & 0x7F) == 0x7F] = 0x7E
    b = _bytes(g, n, k // 2)
    s, bs = _bytes(g, m, k // 32, lo=100, hi=150), _bytes(g, n, k // 32, lo=100, hi=150)
    y = fb.mxfp4_gemm(a, s, "e4m3", b, bs, out_dtype=dtype)
    _near(y, _rows(a, s, "e4m3"), _matrix(b, bs), k, "e4m3", dtype)


@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
@pytest.mark.parametrize("m", [4, 300])
def test_nan_scales_and_codes_stay_in_their_rows(elem, m):
    a, s, b, bs = _grid(_gen(8), m, 80, 256, elem)
    s[1, 3] = 255
    bs[5, 0] = 255
    if elem == "e4m3":
        a.view(torch.uint8)[2, 200] = 0x7F
    for dtype in (torch.float32, torch.bfloat16):
        y = fb.mxfp4_gemm(a, s, elem, b, bs, out_dtype=dtype)
        nan = torch.zeros_like(y, dtype=torch.bool)
        nan[1], nan[:, 5] = True, True
        if elem == "e4m3":
            nan[2] = True
        assert torch.equal(torch.isnan(y), nan)


def _offsets(sizes, behind=0):
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    return torch.from_numpy(off).cuda(), int(off[-1]) + behind


GROUPS = [([5], 0), ([0, 0, 3], 2), ([1] * 9 + [0] * 4, 0), ([300, 0, 7, 64, 1], 5), ([129, 128, 127, 0, 16], 0),
          ([0, 0], 4), ([1000, 3], 1), ([2] * 60, 0), ([33, 17, 0, 500, 64, 256, 31], 3)]


@pytest.mark.parametrize("sizes,behind", GROUPS)
@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_exact(sizes, behind, elem, gather):
    print(f"[mx gemm] groups {sizes[:8]} behind {behind} {elem} gather {gather}", flush=True)
    g = _gen(len(sizes) + behind)
    n, k = (264, 384) if len(sizes) < 20 else (130, 256)
    off, total = _offsets(sizes, behind)
    rows = max(1, total // 3) if gather else total
    a, s, b, bs = _grid(g, rows, n, k, elem, groups=len(sizes))
    index = torch.randint(0, rows, (total,), device="cuda", generator=g, dtype=torch.int32) if gather else None
    at = index.long() if gather else torch.arange(total, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((total, n), float("nan"), dtype=dtype, device="cuda")
        fb.fp8_mxfp4_grouped_gemm(a, s, elem, index, b, bs, off, y)
        x, w, lo = _rows(a, s, elem), _matrix(b, bs), 0
        for e, size in enumerate(sizes):
            assert torch.equal(y[lo:lo + size], (x[at[lo:lo + size]] @ w[e].T).to(dtype)), (e, dtype)
            lo += size
        assert torch.isnan(y[lo:]).all()               # rows behind the last stay


def test_offsets_and_indices_out_of_range_are_clamped():
    """Offsets that fall or pass the rows, indices of any value: no access outside, rows of proper groups right."""
    g = _gen(3)
    a, s, b, bs = _grid(g, 20, 96, 256, "e2m1", groups=4)
    off = torch.tensor([0, 12, 9, 2000000000, -5], dtype=torch.int32, device="cuda")
    index = torch.full((50,), 7, dtype=torch.int32, device="cuda")
    index[3], index[4], index[5] = -9, 2000000000, 19
    y = torch.zeros((50, 96), dtype=torch.float32, device="cuda")
    fb.fp8_mxfp4_grouped_gemm(a, s, "e2m1", index, b, bs, off, y)
    x, w = _rows(a, s, "e2m1"), _matrix(b, bs)
    assert torch.equal(y[:9], (x[index[:9].long().clamp(0, 19)] @ w[0].T).float())     # rows 9 on belong to two groups
    torch.cuda.synchronize()


def test_many_groups_and_large_offsets_of_weights():
    """1024 groups; the last matrices lie more than 4 GiB behind the first."""
    g = _gen(4)
    groups, n, k = 1024, 2048, 4096
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[1:3], off[3:1023], off[1023:] = 2, 5, 9
    b = _bytes(g, 64, n, k // 2).repeat(16, 1, 1)
    bs = _bytes(g, 64, n, k // 32, lo=126, hi=129).repeat(16, 1, 1)
    assert b.numel() == 4 << 30
    a, s, _, _ = _grid(g, 9, 32, k, "e2m1")
    y = fb.mxfp4_grouped_gemm(a, s, "e2m1", b, bs, off, out_dtype=torch.float32)
    x = _rows(a, s, "e2m1")
    for e, lo, hi in ((0, 0, 2), (2, 2, 5), (1022, 5, 9)):
        assert torch.equal(y[lo:hi], (x[lo:hi] @ _matrix(b[e], bs[e]).T).float()), e


def test_rows_do_not_depend_on_other_rows():
    """Rows alone and in a batch of the same launch shape, and repeated calls, give the same bytes."""
    a, s, b, bs = _random(_gen(5), 300, 384, 1024, "e4m3")
    y = fb.mxfp4_gemm(a, s, "e4m3", b, bs)
    assert torch.equal(y, fb.mxfp4_gemm(a, s, "e4m3", b, bs))
    p = torch.randperm(300, device="cuda", generator=_gen(6))
    z = fb.mxfp4_gemm(a.view(torch.uint8)[p], s[p], "e4m3", b, bs)
    assert torch.equal(z, y[p])


@pytest.mark.parametrize("m,n,k,elem,dtype", [
    (8192, 8192, 128, "e4m3", torch.bfloat16), (8192, 8192, 384, "e2m1", torch.bfloat16),
    (8100, 8200, 640, "e4m3", torch.bfloat16), (8192, 8192, 1152, "e2m1", torch.float32),
    (4200, 8194, 896, "e4m3", torch.float32), (8192, 8190, 1024, "e2m1", torch.bfloat16),
    (4096, 8192, 1664, "e4m3", torch.float32)])
def test_many_tiles_of_every_length(m, n, k, elem, dtype):
    """Several tiles for each workgroup: whole ones, cut ones and odd widths follow each other."""
    g = _gen(m + n + k)
    a, s, b, bs = _grid(g, m, n, k, elem)
    y = torch.empty(m, n, dtype=dtype, device="cuda")
    fb.fp8_mxfp4_gemm(a, s, elem, b, bs, y)
    want = _rows(a, s, elem) @ _matrix(b, bs).T
    assert torch.equal(y, want.to(torch.float32).to(dtype))


@pytest.mark.parametrize("elem,gather", [("e4m3", False), ("e4m3", True), ("e2m1", True)])
def test_many_grouped_tiles(elem, gather):
    """Groups of a few tiles each, whole and cut, empty ones between, and rows behind the last group."""
    groups, n, k, behind = 40, 2048, 640, 5
    sizes = [(0, 1, 130, 256, 512, 700, 33, 384)[i % 8] for i in range(groups)]
    total = sum(sizes) + behind
    g = _gen(groups)
    rows = 600 if gather else total
    a, s, b, bs = _grid(g, rows, n, k, elem, groups)
    index = torch.randint(0, rows, (total,), device="cuda", generator=g, dtype=torch.int32) if gather else None
    offsets = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32, device="cuda")
    y = torch.full((total, n), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8_mxfp4_grouped_gemm(a, s, elem, index, b, bs, offsets, y)
    x = _rows(a, s, elem)
    x = x[index.long()] if gather else x
    at = 0
    for e, size in enumerate(sizes):
        want = (x[at:at + size] @ _matrix(b[e], bs[e]).T).to(torch.float32).to(torch.bfloat16)
        assert torch.equal(y[at:at + size], want), e
        at += size
    assert bool((y[at:] == 7.0).all())


@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
def test_rows_past_32_bits(elem):
    """Few rows, the last of them 4 GiB and more into the operand; ones at a few places of each row."""
    k, n = 1 << 24, 16
    m = 262 if elem == "e4m3" else 518
    g = _gen(7)
    q = torch.zeros((m, k if elem == "e4m3" else k // 2), dtype=torch.uint8, device="cuda")
    places = torch.randint(0, k // 2, (m, 8), device="cuda", generator=g) * 2      # even: the low half of an E2M1 byte
    places[:, 7] = k - 2
    one = 0x38 if elem == "e4m3" else 0x02
    q.scatter_(1, places if elem == "e4m3" else places // 2, one)
    a = q.view(torch.float8_e4m3fn) if elem == "e4m3" else q
    s = torch.full((m, k // 32), 127, dtype=torch.uint8, device="cuda")
    b = _bytes(g, n, k // 2)
    bs = torch.full((n, k // 32), 127, dtype=torch.uint8, device="cuda")
    y = torch.empty(m, n, dtype=torch.float32, device="cuda")
    fb.fp8_mxfp4_gemm(a, s, elem, b, bs, y)
    for r in (0, 1, 127, 255, 256, 257, m - 6, m - 1):
        p = torch.unique(places[r])
        want = E2M1.to("cuda")[(b[:, p // 2] & 15).long()].sum(1)
        assert torch.equal(y[r].to(F64), want), r
