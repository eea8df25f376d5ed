"""The ends of the scales' range in the MXFP4 products, and values below the normal range in them and in the gradients.

Values lie on a coarse binary grid under scales a factor of four apart, so that every sum that stays in the fp32 range is
exact (fp32's values below the normal range included: the last bit of every product here is 2^-140 or more, or the whole
sum is below 2^-200 and rounds to zero) and results are equal, bit for bit.  What leaves the range is not finite.
"""

import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from tests.test_gpu_mx_gemm import F64, _bytes, _gen, _matrix, _offsets, _rows

pytestmark = pytest.mark.gpu
LOW, HIGH, ONE, ROOT = (0, 3), (252, 255), (126, 129), (60, 63)       # ROOT: two of them make values below 2^-126


def _rows_of(g, m, k, elem):
    return _bytes(g, m, k // 2) if elem == "e2m1" else (_bytes(g, m, k, hi=9).float() - 4).to(torch.float8_e4m3fn)


@pytest.mark.parametrize("ra,rb", [(LOW, HIGH), (HIGH, LOW), (LOW, ONE), (ONE, LOW), (LOW, LOW), (ROOT, ROOT)])
@pytest.mark.parametrize("m,n", [(4, 40), (20, 9000), (200, 300), (1000, 1100)])
@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
def test_products(ra, rb, m, n, elem):
    print(f"[mx scales] {m}x{n} {elem} {ra} {rb}", flush=True)
    g, k = _gen(m + n + ra[0] + rb[1]), 384
    a, b = _rows_of(g, m, k, elem), _bytes(g, n, k // 2)
    s, bs = _bytes(g, m, k // 32, lo=ra[0], hi=ra[1]), _bytes(g, n, k // 32, lo=rb[0], hi=rb[1])
    want = _rows(a, s, elem) @ _matrix(b, bs).T
    for dtype in (torch.float32, torch.bfloat16):
        y = fb.mxfp4_gemm(a, s, elem, b, bs, out_dtype=dtype)
        assert torch.equal(y, want.float().to(dtype)), dtype
    off, _ = _offsets([m // 2, 0, m - m // 2])
    mats = (b.expand(3, -1, -1).contiguous(), bs.expand(3, -1, -1).contiguous())
    assert torch.equal(fb.mxfp4_grouped_gemm(a, s, elem, *mats, off, out_dtype=torch.float32), want.float())


@pytest.mark.parametrize("m", [4, 300])
@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
def test_zeros_and_what_leaves_the_range(m, elem):
    """Zeros stay zeros under the largest scales; products past the range are infinite with their sign, and those of
    other rows and columns are as they were."""
    n, k = 72, 256
    a, b = torch.zeros(m, k), torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda")
    a[1, 5], a[2, 5] = 1.0, -1.0
    b[3, 2] = 0x20                                       # place 5: 1.0
    s, bs = (torch.full((r, k // 32), 254, dtype=torch.uint8, device="cuda") for r in (m, n))
    if elem == "e4m3":
        q = a.to(torch.float8_e4m3fn).cuda()
    else:
        codes = torch.where(a > 0, 2, torch.where(a < 0, 10, 0)).to(torch.uint8)
        q = (codes[:, 0::2] | (codes[:, 1::2] << 4)).cuda()
    want = torch.zeros(m, n, device="cuda")
    want[1, 3], want[2, 3] = float("inf"), -float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(fb.mxfp4_gemm(q, s, elem, b, bs, out_dtype=dtype), want.to(dtype)), dtype


@pytest.mark.parametrize("m,n", [(1, 64), (3, 9000), (7, 300), (40, 300)])
@pytest.mark.parametrize("scales,size", [(LOW, 1.0), (LOW, 2.0 ** 100), ((220, 250), 2.0 ** -130), (HIGH, 2.0 ** -20)])
def test_bf16_rows(m, n, scales, size):
    """Weights and rows below bf16's normal range, and weights past it (which are infinite, as dequantized ones are).  One
    element of each row is not zero, so nothing is added; an infinite weight beside a zero is a NaN."""
    g, k = _gen(m + n), 64
    q, s = _bytes(g, n, k // 2), _bytes(g, n, k // 32, lo=scales[0], hi=scales[1])
    x = torch.zeros((m, k), device="cuda")
    for i in range(m):
        x[i, (9 * i + 3) % k] = size
    x = x.to(torch.bfloat16)
    assert torch.all((x != 0).sum(1) == 1)
    w = fb.mxfp4_dequantize(q, s).to(F64)
    assert torch.equal(w.abs() == float("inf"), _matrix(q, s).abs() >= 2.0 ** 128)
    want = x.to(F64) @ torch.nan_to_num(w, posinf=0.0, neginf=0.0).T
    past = (w.abs() == float("inf")).to(F64)
    at = (x != 0).to(F64) @ past.T              # the row's own element meets an infinite weight
    nan = past.sum(1)[None] - at > 0                                    # another one does: 0 times infinity
    y = fb.mxfp4_matvec(x, q, s, out_dtype=torch.float32)
    assert torch.equal(torch.isnan(y), nan)
    assert torch.all(y[~nan & (at > 0)].abs() == float("inf"))
    rest = ~nan & (at == 0)
    assert torch.equal(y[rest], want[rest].float())
    yg = fb.mxfp4_grouped_matvec(x, q[None], s[None], torch.tensor([0, m], dtype=torch.int32, device="cuda"),
                                 out_dtype=torch.float32)
    assert torch.equal(torch.isnan(yg), nan) and torch.equal(yg[~nan], y[~nan])


@pytest.mark.parametrize("rows,n,k", [(20, 64, 72), (300, 2048, 4096)])
def test_gradients_below_the_normal_range(rows, n, k):
    """dy of 2^-130 (times small integers) and rows and weights of 2^20: exact, as larger ones are."""
    g = _gen(rows)

    def ints(*shape):
        return torch.randint(-4, 5, shape, device="cuda", generator=g).float()

    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    dy, w, x = ((v * f).to(torch.bfloat16) for v, f in
                ((ints(rows, n), 2.0 ** -130), (ints(1, n, k), 2.0 ** 20), (ints(rows, k), 2.0 ** 20)))
    d = dy.to(F64)
    assert torch.equal(fb.grouped_dgrad(dy, w, off, out_dtype=torch.float32), (d @ w[0].to(F64)).float())
    assert torch.equal(fb.grouped_wgrad(dy, x, off)[0], (d.T @ x.to(F64)).float())
