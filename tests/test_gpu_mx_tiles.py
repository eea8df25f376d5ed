"""Every tile that fp8_mxfp4_gemm and fp8_mxfp4_grouped_gemm choose, by sizes that lead to it on 256 CUs: cut rows and
columns, a last half stage of K, and more than one tile for each workgroup where the choice allows it.  Values on a coarse
binary grid make every sum exact in fp32, so results are equal, bit for bit.

Tiles are named rows x columns / waves; `to` gives those of E2M1 rows, of E4M3 rows with bf16 and with float results.
"""

import numpy as np
import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from tests.test_gpu_mx_gemm import _gen, _grid, _matrix, _offsets, _rows

pytestmark = pytest.mark.gpu
KINDS = [("e2m1", torch.bfloat16), ("e2m1", torch.float32), ("e4m3", torch.bfloat16), ("e4m3", torch.float32)]

DENSE = [  # m, n, k, to
    (1000, 16390, 384, "128x256/8, 128x256/8, 64x256/8"),
    (1100, 10242, 384, "256x256/4, 128x256/8, 64x256/8"),
    (4100, 8194, 640, "256x256/4, 128x256/8, 128x256/8"),
    (2050, 2594, 640, "128x128/8, 128x128/8, 64x256/8"),
    (512, 4098, 384, "64x64/4, 64x64/4, 32x128/4"),
    (630, 4830, 640, "64x64/4, 64x64/4, 32x128/4"),
    (60, 49002, 384, "64x256/8, 64x256/8, 64x256/8"),
    (30, 24578, 384, "32x128/4, 32x128/4, 32x128/4"),
    (30, 70002, 128, "32x128/4, 32x128/4, 32x128/4"),
    (30, 8330, 640, "64x64/8, 64x64/8, 32x128/4"),
    (300, 1030, 896, "64x64/8, 64x64/8, 32x128/4"),
]


@pytest.mark.parametrize("m,n,k,to", DENSE)
@pytest.mark.parametrize("elem,dtype", KINDS)
def test_dense(m, n, k, to, elem, dtype):
    print(f"[mx tiles] {m}x{n}x{k} {elem} {dtype}: {to}", flush=True)
    a, s, b, bs = _grid(_gen(m + n + k), m, n, k, elem)
    y = torch.full((m, n), float("nan"), dtype=dtype, device="cuda")
    fb.fp8_mxfp4_gemm(a, s, elem, b, bs, y)
    assert torch.equal(y, (_rows(a, s, elem) @ _matrix(b, bs).T).to(dtype))


def _cycle(pattern, groups):
    return [pattern[i % len(pattern)] for i in range(groups)]


GROUPED = [  # sizes, n, k, to
    (_cycle((31, 0, 64, 1, 33, 70, 0, 32), 64), 4098, 384, "32x128/4, 32x128/4, 32x128/4"),
    (_cycle((64, 0, 130, 1, 65, 50), 48), 2050, 640, "64x256/8, 64x256/8, 64x256/8"),
    ([500, 700, 0, 513, 1, 640, 900, 260], 1270, 384, "128x128/8, 128x128/8, 64x256/8"),
    ([65, 190, 0, 64, 1, 129, 300, 33, 100, 120], 2430, 384, "64x64/4, 64x64/4, 64x256/8"),
    ([70, 1, 0, 90, 65], 200, 640, "64x64/8, 64x64/8, 32x128/4"),
    ([1300, 1025, 0, 2100], 2562, 384, "256x256/4, 128x256/8, 64x256/8"),
    (_cycle((300, 257, 0, 640), 40), 2306, 384, "128x256/8, 128x256/8, 128x256/8"),
]


@pytest.mark.parametrize("sizes,n,k,to", GROUPED)
@pytest.mark.parametrize("elem,dtype", KINDS)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(sizes, n, k, to, elem, dtype, gather):
    print(f"[mx tiles] {len(sizes)} groups {sizes[:6]} {n}x{k} {elem} {dtype} gather {gather}: {to}", flush=True)
    g = _gen(len(sizes) + n)
    off, total = _offsets(sizes, 3)
    rows = 333 if gather else total
    a, s, b, bs = _grid(g, rows, n, k, elem, groups=len(sizes))
    index = torch.randint(0, rows, (total,), device="cuda", generator=g, dtype=torch.int32) if gather else None
    y = torch.full((total, n), float("nan"), dtype=dtype, device="cuda")
    fb.fp8_mxfp4_grouped_gemm(a, s, elem, index, b, bs, off, y)
    x, ends = _rows(a, s, elem), np.cumsum(sizes)
    x = x[index.long()] if gather else x
    for e, (size, end) in enumerate(zip(sizes, ends)):
        assert torch.equal(y[end - size:end], (x[end - size:end] @ _matrix(b[e], bs[e]).T).to(dtype)), e
    assert torch.isnan(y[int(ends[-1]):]).all()
