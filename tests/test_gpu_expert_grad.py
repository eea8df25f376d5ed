"""GPU parity of fp8_grouped_dgrad / fp8_grouped_wgrad with float64 products, the formula's by autograd and by differences.

Values on a coarse binary grid give exact sums whatever their order; random values are off by at most (terms) 2^-24 of the
sum of magnitudes and a bf16 result by 2^-8 of the value more.
"""

import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from tests.test_gpu_mx_gemm import F64, GROUPS, _gen, _offsets

pytestmark = pytest.mark.gpu


def _small(g, *shape):
    return torch.randint(-4, 5, shape, device="cuda", generator=g).to(torch.bfloat16)


def _index(g, rows, total, gather):
    if not gather:
        return None, torch.arange(total, device="cuda")
    i = torch.randint(0, rows, (total,), device="cuda", generator=g, dtype=torch.int32)
    return i, i.long()


SIZES = [(8, 8), (64, 264), (264, 72), (1000, 520), (136, 1032)]


@pytest.mark.parametrize("sizes,behind", GROUPS)
@pytest.mark.parametrize("n,k", SIZES)
def test_dgrad_exact(sizes, behind, n, k):
    print(f"[dgrad] groups {sizes[:8]} behind {behind} {n}x{k}", flush=True)
    g = _gen(n + k)
    off, total = _offsets(sizes, behind)
    dy, w = _small(g, total, n), _small(g, len(sizes), n, k)
    for dtype in (torch.float32, torch.bfloat16):
        dx = torch.full((total, k), float("nan"), dtype=dtype, device="cuda")
        fb.fp8_grouped_dgrad(dy, w, off, dx)
        lo = 0
        for e, size in enumerate(sizes):
            assert torch.equal(dx[lo:lo + size], (dy[lo:lo + size].to(F64) @ w[e].to(F64)).to(dtype)), (e, dtype)
            lo += size
        assert torch.isnan(dx[lo:]).all()


@pytest.mark.parametrize("sizes,behind", GROUPS)
@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("gather", [False, True])
def test_wgrad_exact(sizes, behind, n, k, gather):
    print(f"[wgrad] groups {sizes[:8]} behind {behind} {n}x{k} gather {gather}", flush=True)
    g = _gen(n + k + gather)
    off, total = _offsets(sizes, behind)
    rows = max(1, total // 3) if gather else total
    dy, x = _small(g, total, n), _small(g, rows, k)
    index, at = _index(g, rows, total, gather)
    for dtype in (torch.float32, torch.bfloat16):
        dw = torch.full((len(sizes), n, k), float("nan"), dtype=dtype, device="cuda")
        fb.fp8_grouped_wgrad(dy, x, index, off, dw)
        lo = 0
        for e, size in enumerate(sizes):
            want = dy[lo:lo + size].to(F64).T @ x[at[lo:lo + size]].to(F64)
            assert torch.equal(dw[e], want.to(dtype)), (e, dtype)
            lo += size


@pytest.mark.parametrize("sizes,n,k", [([700, 0, 45, 300], 520, 712), ([2000], 256, 256), ([31, 33], 4096, 328)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_random(sizes, n, k, dtype):
    print(f"[grads] random {sizes} {n}x{k} {dtype}", flush=True)
    g = _gen(n * k)
    off, total = _offsets(sizes)
    dy = (1e-3 * torch.randn((total, n), device="cuda", generator=g)).to(torch.bfloat16)
    x = torch.randn((total, k), device="cuda", generator=g).to(torch.bfloat16)
    w = (0.02 * torch.randn((len(sizes), n, k), device="cuda", generator=g)).to(torch.bfloat16)
    index = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    dx = fb.grouped_dgrad(dy, w, off, out_dtype=dtype)
    dw = fb.grouped_wgrad(dy, x, off, row_index=index, out_dtype=dtype)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    lo = 0
    for e, size in enumerate(sizes):
        d, xr, we = dy[lo:lo + size].to(F64), x[index[lo:lo + size].long()].to(F64), w[e].to(F64)
        for got, a, b, terms in ((dx[lo:lo + size], d, we, n), (dw[e], d.T, xr, size)):
            want, mag = a @ b, a.abs() @ b.abs()
            assert torch.all((got.to(F64) - want).abs() <= terms * 2.0 ** -24 * mag + half * want.abs()), e
        lo += size


def test_against_autograd_of_the_forward_product():
    """Through y = x[index] . W^T of the forward call's own decoded weights, in float64."""
    g = _gen(11)
    sizes, n, k = [40, 0, 25], 128, 256
    off, total = _offsets(sizes)
    w = (0.1 * torch.randn((3 * n, k), device="cuda", generator=g)).to(torch.bfloat16)
    q, s, wdq = fb.mxfp4_quantize(w, dequant=True)
    x = torch.randn((30, k), device="cuda", generator=g).to(torch.bfloat16)
    a, a_scale, xdq = fb.quantize(x, "1x32", dequant=True)
    index = torch.randint(0, 30, (total,), device="cuda", generator=g, dtype=torch.int32)
    y = fb.mxfp4_grouped_gemm(a, a_scale, "e4m3", q.view(3, n, k // 2), s.view(3, n, k // 32), off, row_index=index,
                              out_dtype=torch.float32)
    xr = xdq.to(F64).requires_grad_(True)
    wr = wdq.view(3, n, k).to(F64).requires_grad_(True)
    rows, lo = [], 0
    for e, size in enumerate(sizes):
        rows.append(xr[index[lo:lo + size].long()] @ wr[e].T)
        lo += size
    ref = torch.cat(rows)
    assert (y.to(F64) - ref).norm() <= 1e-6 * ref.norm()
    dy = torch.randn((total, n), device="cuda", generator=g).to(torch.bfloat16)
    gx, gw = torch.autograd.grad(ref, (xr, wr), dy.to(F64))
    dx = fb.grouped_dgrad(dy, wdq.view(3, n, k), off, out_dtype=torch.float32)
    dw = fb.grouped_wgrad(dy, xdq, off, row_index=index)
    mine = torch.zeros_like(gx).index_add_(0, index.long(), dx.to(F64))     # rows read more than once collect all
    assert (mine - gx).norm() <= 1e-6 * gx.norm() and (dw.to(F64) - gw).norm() <= 1e-6 * gw.norm()


def test_against_differences():
    """Central differences of sum(dy * y) along random directions: y is linear in x and in W, so a step of any size
    gives the derivative; operands on a binary grid keep it exact."""
    g = _gen(12)
    sizes, n, k = [9, 20], 64, 128
    off, total = _offsets(sizes)
    dy, x, w = _small(g, total, n), _small(g, total, k), _small(g, 2, n, k)
    dx = fb.grouped_dgrad(dy, w, off, out_dtype=torch.float32).to(F64)
    dw = fb.grouped_wgrad(dy, x, off).to(F64)

    def loss(x, w):
        return sum((dy[lo:hi].to(F64) * (x[lo:hi] @ w[e].T)).sum() for e, (lo, hi) in enumerate(((0, 9), (9, 29))))

    for i in range(4):
        u, v = _small(g, total, k).to(F64), _small(g, 2, n, k).to(F64)
        d = (loss(x.to(F64) + u, w.to(F64)) - loss(x.to(F64) - u, w.to(F64))) / 2
        assert d == (dx * u).sum()
        d = (loss(x.to(F64), w.to(F64) + v) - loss(x.to(F64), w.to(F64) - v)) / 2
        assert d == (dw * v).sum()


def test_infinities_and_nan_stay_in_their_rows():
    """A row that is not finite reaches its own dx, and the dw of its own group only; rows of other groups and rows
    behind the last are not read."""
    g = _gen(13)
    sizes, n, k = [20, 13, 40], 72, 136
    off, total = _offsets(sizes, 3)
    dy, x, w = _small(g, total, n), _small(g, total, k), _small(g, 3, n, k)
    clean_dx, clean_dw = fb.grouped_dgrad(dy, w, off), fb.grouped_wgrad(dy, x, off)
    dy[25], x[28] = float("nan"), float("inf")
    dy[total - 3:], x[total - 3:] = float("nan"), float("nan")
    dx, dw = fb.grouped_dgrad(dy, w, off), fb.grouped_wgrad(dy, x, off)
    keep = [i for i in range(total) if i != 25]
    assert torch.isnan(dx[25]).all() and torch.equal(dx[keep], clean_dx[keep])
    assert not torch.isfinite(dw[1]).any() and torch.equal(dw[[0, 2]], clean_dw[[0, 2]])
    w2 = w.clone()
    w2[2] = float("nan")
    dx = fb.grouped_dgrad(dy, w2, off)
    assert torch.isnan(dx[33:73]).all() and torch.equal(dx[:25], clean_dx[:25])


def test_no_rows_no_columns_and_clamped_offsets():
    g = _gen(14)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    dw = fb.grouped_wgrad(e, torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"), off)
    assert dw.shape == (3, 64, 32) and not dw.any()
    assert fb.grouped_dgrad(e, _small(g, 3, 64, 32), off).shape == (0, 32)
    off[1:] = torch.tensor([5, 5, 9], dtype=torch.int32)
    dx = torch.full((9, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8_grouped_dgrad(_small(g, 9, 0), _small(g, 3, 0, 32), off, dx)
    assert not dx.any()
    off = torch.tensor([0, 12, 9, 2000000000, -5], dtype=torch.int32, device="cuda")
    dy, w, x = _small(g, 50, 64), _small(g, 4, 64, 40), _small(g, 20, 40)
    index = torch.full((50,), 7, dtype=torch.int32, device="cuda")
    index[3], index[4], index[5] = -9, 2000000000, 19
    dx = fb.grouped_dgrad(dy, w, off, out_dtype=torch.float32)
    assert torch.equal(dx[:9], (dy[:9].to(F64) @ w[0].to(F64)).float())       # rows 9 on belong to two groups
    dw = fb.grouped_wgrad(dy, x, off, row_index=index)
    at = index.long().clamp(0, 19)
    assert torch.equal(dw[0], (dy[:12].to(F64).T @ x[at[:12]].to(F64)).float()) and not dw[1].any() and not dw[3].any()


def test_large_weights_and_many_groups():
    """Weights whose last matrix lies past 4 GiB, groups enough to fill the table."""
    g = _gen(15)
    n, k, groups = 2048, 2048, 1024
    w = torch.zeros((groups, n, k), dtype=torch.bfloat16, device="cuda")
    w[0], w[600], w[1023] = _small(g, n, k), _small(g, n, k), _small(g, n, k)
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[1:601], off[601:1024], off[1024] = 3, 10, 50
    dy, x = _small(g, 50, n), _small(g, 50, k)
    dx = fb.grouped_dgrad(dy, w, off, out_dtype=torch.float32)
    for e, lo, hi in ((0, 0, 3), (600, 3, 10), (1023, 10, 50)):
        assert torch.equal(dx[lo:hi], (dy[lo:hi].to(F64) @ w[e].to(F64)).float()), e
    dw = torch.full((groups, n, k), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8_grouped_wgrad(dy, x, None, off, dw)
    for e, lo, hi in ((0, 0, 3), (600, 3, 10), (1023, 10, 50)):
        assert torch.equal(dw[e], (dy[lo:hi].to(F64).T @ x[lo:hi].to(F64)).to(torch.bfloat16)), e
    for e in (1, 599, 601, 1022):
        assert not dw[e].any()


@pytest.mark.parametrize("n,k", [(1024, 2048), (1032, 2040)])
@pytest.mark.parametrize("gather", [False, True])
def test_many_tiles(n, k, gather):
    """Several tiles for each workgroup: whole and cut ones, groups of no, one and many stages in turn."""
    sizes = [(0, 300, 1, 64, 0, 0, 130, 513, 65, 256)[i % 10] for i in range(43)]
    g = _gen(n + gather)
    off, total = _offsets(sizes, 3)
    rows = 500 if gather else total
    dy, x, w = _small(g, total, n), _small(g, rows, k), _small(g, len(sizes), n, k)
    index, at = _index(g, rows, total, gather)
    for dtype in (torch.float32, torch.bfloat16):
        dx = torch.full((total, k), float("nan"), dtype=dtype, device="cuda")
        dw = torch.full((len(sizes), n, k), float("nan"), dtype=dtype, device="cuda")
        fb.fp8_grouped_dgrad(dy, w, off, dx)
        fb.fp8_grouped_wgrad(dy, x, index, off, dw)
        lo = 0
        for e, size in enumerate(sizes):
            d = dy[lo:lo + size].to(F64)
            assert torch.equal(dx[lo:lo + size], (d @ w[e].to(F64)).to(dtype)), (e, dtype)
            assert torch.equal(dw[e], (d.T @ x[at[lo:lo + size]].to(F64)).to(dtype)), (e, dtype)
            lo += size
        assert torch.isnan(dx[lo:]).all()


@pytest.mark.parametrize("n,k", [(72, 136), (2048, 4096)])
@pytest.mark.parametrize("gather", [False, True])
def test_bf16_weights_without_rows_and_with_nan(n, k, gather):
    """No rows at all give zeros; what is not finite reaches its own group's matrix only."""
    g = _gen(15)
    e = torch.empty((0, n), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((3, n, k), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8_grouped_wgrad(e, torch.empty((0, k), dtype=torch.bfloat16, device="cuda"), None,
                         torch.zeros(4, dtype=torch.int32, device="cuda"), dw)
    assert not dw.any()
    off, total = _offsets([20, 13, 0, 140], 3)
    dy, x = _small(g, total, n), _small(g, total, k)
    index = torch.arange(total, device="cuda", dtype=torch.int32) if gather else None
    clean = fb.grouped_wgrad(dy, x, off, row_index=index, out_dtype=torch.bfloat16)
    dy[25], x[28] = float("nan"), float("inf")
    dy[total - 3:], x[total - 3:] = float("nan"), float("nan")
    dw = fb.grouped_wgrad(dy, x, off, row_index=index, out_dtype=torch.bfloat16)
    assert not torch.isfinite(dw[1]).any() and torch.equal(dw[[0, 2, 3]], clean[[0, 2, 3]])
