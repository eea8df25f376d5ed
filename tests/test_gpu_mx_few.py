"""Few quantized rows, gathered: every wave of the kernel that cuts K walks several stages, whose scales are read from the
gathered rows.  Values on a coarse binary grid make every sum exact in fp32, so results are equal, bit for bit."""

import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from tests.test_gpu_mx_gemm import _gen, _grid, _matrix, _offsets, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes,n,k", [([1], 40, 2688), ([2, 0, 3, 1, 9, 0], 70, 4224), ([1] * 20 + [17], 33, 2176),
                                       ([4, 5, 30, 0, 1, 0, 0, 2], 2050, 1920), ([3, 0, 4], 130, 7168),
                                       ([3, 1, 0, 2, 17, 1, 5, 0, 4, 1, 1, 8], 4100, 1664)])
@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gathered_rows_over_many_stages(sizes, n, k, elem, dtype):
    print(f"[mx few] {sizes} {n}x{k} {elem} {dtype}", flush=True)
    g = _gen(n + k)
    off, total = _offsets(sizes, 2)
    rows = 11
    a, s, b, bs = _grid(g, rows, n, k, elem, groups=len(sizes))
    index = torch.randint(0, rows, (total,), device="cuda", generator=g, dtype=torch.int32)
    index[0], index[total - 3] = rows - 1, 0
    y = torch.full((total, n), float("nan"), dtype=dtype, device="cuda")
    fb.fp8_mxfp4_grouped_gemm(a, s, elem, index, b, bs, off, y)
    x, w, lo = _rows(a, s, elem)[index.long()], _matrix(b, bs), 0
    for e, size in enumerate(sizes):
        assert torch.equal(y[lo:lo + size], (x[lo:lo + size] @ w[e].T).to(dtype)), e
        lo += size
    assert torch.isnan(y[lo:]).all()
