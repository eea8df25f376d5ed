"""GPU parity of the MXFP4 codec against the oracle: every byte equal.  The quotient x 2^-X is exact, so nothing is
left to a tolerance."""

import numpy as np
import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from oracle import mxfp4
from oracle.codec import f32_to_bf16
from tests.gpu_helpers import assert_bytes_equal, bf16_from_bits
from workloads import bf16_bits, normal_bf16

pytestmark = pytest.mark.gpu


def _check(bits, rule):
    q, s, dq = fb.mxfp4_quantize(bf16_from_bits(bits), rule, dequant=True)
    oq, os_, odq = mxfp4.quantize(bits, rule)
    assert_bytes_equal(s.cpu().numpy(), os_, "scales")
    assert_bytes_equal(q.cpu().numpy(), oq, "codes")
    assert_bytes_equal(bf16_bits(dq), odq, "fake-quant values")
    q2, s2 = fb.mxfp4_quantize(bf16_from_bits(bits), rule)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert_bytes_equal(bf16_bits(fb.mxfp4_dequantize(q, s)), odq, "dequantized values")


@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (3, 96), (17, 4128), (257, 64), (64, 2048), (1000, 160), (5, 32768)])
@pytest.mark.parametrize("rule", ["ceil", "floor"])
def test_random(rows, cols, rule):
    print(f"[mxfp4] {rows}x{cols} {rule}", flush=True)
    x = normal_bf16((rows, cols), 1.0, rows + cols, outlier_frac=0.01, outlier_mult=100.0)
    _check(bf16_bits(x), rule)


@pytest.mark.parametrize("rule", ["ceil", "floor"])
def test_every_value_in_every_binade(rule):
    """Each bf16 value beside a block maximum of its own and the next nine binades (further down it rounds to zero)."""
    rng = np.random.default_rng(1)
    vals = np.arange(0x7F80, dtype=np.uint16)
    rows = []
    for up in (0, 0x20, 0x41, 0x80, 0xC1, 0x140, 0x1C0, 0x240, 0x300, 0x480):
        x = vals.reshape(-1, 30)
        top = np.minimum(x.max(1) + up, 0x7F7F)
        block = np.concatenate([x, top[:, None], np.zeros_like(top)[:, None]], 1).astype(np.uint16)
        rows.append(block)
    bits = np.concatenate(rows) | (rng.integers(0, 2, (sum(len(r) for r in rows), 32)).astype(np.uint16) << 15)
    _check(bits, rule)


@pytest.mark.parametrize("rule", ["ceil", "floor"])
def test_zeros_subnormals_and_the_largest(rule):
    x = np.zeros((9, 64), np.uint16)
    x[1] = 0x8000
    x[2, :32], x[2, 32:] = 0x0001, 0x8001
    x[3, 7], x[3, 40] = 0x007F, 0x0080
    x[4] = 0x7F7F
    x[5, ::2], x[5, 1::2] = 0xFF7F, 0x7F00
    x[6, 3], x[6, 60] = 0x7F40, 0x7F41                 # 6 2^125 and just past it
    x[7] = f32_to_bf16(np.linspace(-7, 7, 64).astype(np.float32))
    x[8, 0], x[8, 1], x[8, 33] = 0x0100, 0x0001, 0x01C0
    _check(x, rule)


def test_every_code_and_scale_dequantized():
    q = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (16, 1))
    s = np.arange(256, dtype=np.uint8)[:, None]
    x = fb.mxfp4_dequantize(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda())
    assert_bytes_equal(bf16_bits(x[:255]), mxfp4.dequantize(q[:255], s[:255]), "values")
    assert torch.isnan(x[255]).all()


def test_empty_and_refused():
    for rows, cols in ((0, 64), (3, 0)):
        q, s, dq = fb.mxfp4_quantize(torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda"), dequant=True)
        assert q.shape == (rows, cols // 2) and fb.mxfp4_dequantize(q, s).shape == (rows, cols)
    with pytest.raises(fb.Fp8Error) as e:
        fb.mxfp4_quantize(torch.zeros((2, 48), dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == 2
    flat = torch.zeros(4 * 32 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fb.Fp8Error) as e:
        fb.mxfp4_quantize(flat[4:].view(4, 32))
    assert e.value.status == 3
