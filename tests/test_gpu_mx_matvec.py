"""GPU parity of fp8_mxfp4_matvec / fp8_mxfp4_grouped_matvec with float64 products of the decoded weights.

Values on a coarse binary grid give exact sums whatever their order; random values are off by at most k 2^-24 of the
sum of magnitudes and a bf16 result by 2^-8 of the value more.
"""

import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from tests.test_gpu_mx_gemm import F64, GROUPS, _bytes, _gen, _matrix, _near, _offsets

pytestmark = pytest.mark.gpu


def _grid(g, m, n, k, groups=None):
    q = _bytes(g, *(() if groups is None else (groups,)), n, k // 2)
    s = _bytes(g, *q.shape[:-1], k // 32, lo=126, hi=129)
    return (_bytes(g, m, k, hi=17).float() - 8).to(torch.bfloat16), q, s


SHAPES = [(1, 1, 32), (1, 64, 128), (2, 33, 96), (3, 100, 2048), (16, 48, 256), (17, 31, 288), (33, 64, 512),
          (5, 7, 7200), (1, 257, 4096), (40, 16, 64), (8, 130, 96), (1, 4099, 32), (1, 4112, 320), (2, 5000, 192),
          (9, 5008, 192), (20, 5008, 224), (2, 16400, 64), (1, 16401, 576), (30, 16400, 128), (12, 16400, 96),
          (50, 300, 1024), (31, 4097, 288), (3, 300, 2080), (4, 130, 4096), (5, 520, 2336), (8, 4096, 2048),
          (7, 33, 6176), (32, 4200, 1280), (17, 100, 4160), (29, 90, 2208), (9, 16, 512), (100, 64, 1024),
          (33, 2048, 544), (1000, 40, 256), (17, 2033, 64), (1, 4096, 7168), (2, 8192, 1024), (1, 16384, 4128)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_exact_on_a_grid(m, n, k):
    print(f"[mx matvec] grid {m}x{n}x{k}", flush=True)
    x, q, s = _grid(_gen(m + n + k), m, n, k)
    want = x.to(F64) @ _matrix(q, s).T
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(fb.mxfp4_matvec(x, q, s, out_dtype=dtype), want.to(dtype)), dtype


@pytest.mark.parametrize("m,n,k", [(1, 256, 7168), (2, 4100, 1024), (13, 200, 7200), (32, 64, 2048), (3, 96, 1056)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_random(m, n, k, dtype):
    print(f"[mx matvec] random {m}x{n}x{k} {dtype}", flush=True)
    g = _gen(m + n + k)
    x = torch.randn((m, k), device="cuda", generator=g).to(torch.bfloat16)
    q, s = fb.mxfp4_quantize((0.02 * torch.randn((n, k), device="cuda", generator=g)).to(torch.bfloat16))
    _near(fb.mxfp4_matvec(x, q, s, out_dtype=dtype), x.to(F64), _matrix(q, s), k, "e2m1", dtype)


@pytest.mark.parametrize("m", [1, 2, 7])
@pytest.mark.parametrize("n", [256, 20000])
def test_every_code_and_scale(m, n):
    """Every code under every scale byte whose values bf16 holds as normal numbers; single elements, so sums are
    exact.  Large x beside them: a block's products stay in the fp32 range when their scaled ones do."""
    g = _gen(n + m)
    q = _bytes(g, n, 32)
    s = _bytes(g, n, 2, lo=3, hi=251)
    x = torch.zeros((m, 64), device="cuda")
    for i in range(m):
        x[i, (9 * i + 3) % 64] = 2.0 ** (3 * i - 2)
    want = (x.to(F64) @ _matrix(q, s).T).float()
    y = fb.mxfp4_matvec(x.to(torch.bfloat16), q, s, out_dtype=torch.float32)
    normal = want.abs() >= 2.0 ** -126
    assert torch.equal(y[normal], want[normal]) and torch.all(y[~normal].abs() <= 2.0 ** -126)
    s[:] = _bytes(g, n, 2, lo=30, hi=60)
    x = x * 2.0 ** 100
    y = fb.mxfp4_matvec(x.to(torch.bfloat16), q, s, out_dtype=torch.float32)
    assert torch.equal(y, (x.to(F64) @ _matrix(q, s).T).float())


@pytest.mark.parametrize("m", [1, 3, 20])
@pytest.mark.parametrize("n", [100, 20000])
def test_nan_and_infinity_stay_in_their_rows(m, n):
    x, q, s = _grid(_gen(2), m, n, 128)
    s[5, 1] = 255
    want = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    want[:, 5] = True
    if m > 1:
        x[1, 3] = float("nan")
        want[1] = True
    if m > 2:
        x[2, 0] = float("inf")
    y = fb.mxfp4_matvec(x, q, s, out_dtype=torch.float32)
    if m > 2:
        clean = [i for i in range(m) if i != 2]
        assert torch.equal(torch.isnan(y[clean]), want[clean]) and not torch.isfinite(y[2]).any()
    else:
        assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("sizes,behind", GROUPS)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k", [(100, 416), (4100, 256), (40, 1024)])
def test_grouped_exact(sizes, behind, gather, n, k):
    print(f"[mx matvec] groups {sizes[:8]} behind {behind} gather {gather} {n}x{k}", flush=True)
    g = _gen(len(sizes) + behind)
    off, total = _offsets(sizes, behind)
    rows = max(1, total // 3) if gather else total
    x, q, s = _grid(g, rows, n, k, groups=len(sizes))
    index = torch.randint(0, rows, (total,), device="cuda", generator=g, dtype=torch.int32) if gather else None
    at = index.long() if gather else torch.arange(total, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((total, n), float("nan"), dtype=dtype, device="cuda")
        fb.fp8_mxfp4_grouped_matvec(x, index, q, s, off, y)
        lo = 0
        for e, size in enumerate(sizes):
            want = (x[at[lo:lo + size]].to(F64) @ _matrix(q[e], s[e]).T).to(dtype)
            assert torch.equal(y[lo:lo + size], want), (e, dtype)
            lo += size
        assert torch.isnan(y[lo:]).all()


def test_offsets_and_indices_out_of_range_are_clamped():
    x, q, s = _grid(_gen(3), 20, 96, 256, groups=4)
    off = torch.tensor([0, 12, 9, 2000000000, -5], dtype=torch.int32, device="cuda")
    index = torch.full((50,), 7, dtype=torch.int32, device="cuda")
    index[3], index[4], index[5] = -9, 2000000000, 19
    y = torch.zeros((50, 96), dtype=torch.float32, device="cuda")
    fb.fp8_mxfp4_grouped_matvec(x, index, q, s, off, y)
    want = x[index[:9].long().clamp(0, 19)].to(F64) @ _matrix(q[0], s[0]).T
    assert torch.equal(y[:9], want.float())              # rows 9 on belong to two groups
    torch.cuda.synchronize()


def test_unaligned_results_and_scales():
    """Scales at any byte, results at their element's alignment."""
    x, q, s = _grid(_gen(4), 3, 75, 224)
    sb = torch.zeros(s.numel() + 1, dtype=torch.uint8, device="cuda")
    st = sb[1:].view(s.shape)
    st.copy_(s)
    want = x.to(F64) @ _matrix(q, s).T
    for dtype in (torch.float32, torch.bfloat16):
        yb = torch.zeros(3 * 75 + 1, dtype=dtype, device="cuda")
        y = yb[1:].view(3, 75)
        fb.fp8_mxfp4_matvec(x, q, st, y)
        assert torch.equal(y, want.to(dtype)) and yb[0] == 0
