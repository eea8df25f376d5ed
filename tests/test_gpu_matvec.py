"""GPU parity of fp8_nvfp4_matvec / fp8_nvfp4_grouped_matvec against the oracle.

Two kinds of checks.  Values on a coarse binary grid (integer x, powers of two as scales) make every product and
every partial sum exact in fp32 whatever the order of addition, so results are equal, bit for bit.  Random values:
products are exact and any order of K additions in fp32 is off by at most K 2^-24 of the sum of magnitudes; the tensor
scale and the output add 2^-23, a bf16 output 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from oracle import moe, nvfp4
from oracle.codec import bf16_to_f32, f32_to_bf16
from tests.gpu_helpers import bf16_from_bits
from workloads import bf16_bits

pytestmark = pytest.mark.gpu


def _grid_matrix(rng, rows, k):
    """Codes of any value, scales 2^-2 .. 2^2 as e4m3 codes."""
    q = rng.integers(0, 256, (rows, k // 2)).astype(np.uint8)
    bs = ((rng.integers(-2, 3, (rows, k // 16)) + 7) << 3).astype(np.uint8)
    return q, bs


def _random_matrix(rng, rows, k):
    w = f32_to_bf16((0.02 * rng.standard_normal((rows, k))).astype(np.float32))
    q, bs, gs, _, _ = nvfp4.quantize(w)
    return q, bs, gs


def _out(y):
    return y.double().cpu().numpy() if y.dtype == torch.float32 else bf16_to_f32(bf16_bits(y)).astype(np.float64)


def _bf16(v):
    return bf16_to_f32(f32_to_bf16(v.astype(np.float32))).astype(np.float64)


SHAPES = [(1, 1, 16), (1, 64, 128), (2, 33, 48), (3, 100, 2048), (16, 48, 256), (17, 31, 272), (33, 64, 512),
          (5, 7, 7184), (1, 257, 4096), (40, 16, 64), (8, 130, 96), (1, 4099, 32)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_exact_on_a_grid(m, n, k, dtype):
    print(f"[matvec] grid {m}x{n}x{k} {dtype}", flush=True)
    rng = np.random.default_rng(m * 31 + n + k)
    x = rng.integers(-8, 9, (m, k)).astype(np.float64)
    q, bs = _grid_matrix(rng, n, k)
    gs = np.array([2.0 ** -6], np.float32)
    y = fb.nvfp4_matvec(bf16_from_bits(f32_to_bf16(x.astype(np.float32))), torch.from_numpy(q).cuda(),
                        torch.from_numpy(bs).cuda(), torch.from_numpy(gs).cuda(), out_dtype=dtype)
    want = x @ moe.nvfp4_matrix(q, bs, gs, n).T
    assert np.array_equal(_out(y), want if dtype == torch.float32 else _bf16(want))


@pytest.mark.parametrize("m,n,k", [(1, 256, 7168), (13, 200, 7184), (32, 64, 2048), (3, 96, 1040)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_random(m, n, k, dtype):
    print(f"[matvec] random {m}x{n}x{k} {dtype}", flush=True)
    rng = np.random.default_rng(m + n + k)
    xb = f32_to_bf16(rng.standard_normal((m, k)).astype(np.float32))
    q, bs, gs = _random_matrix(rng, n, k)
    y = fb.nvfp4_matvec(bf16_from_bits(xb), torch.from_numpy(q).cuda(), torch.from_numpy(bs).cuda(),
                        torch.from_numpy(gs).cuda(), out_dtype=dtype)
    x, w = bf16_to_f32(xb).astype(np.float64), moe.nvfp4_matrix(q, bs, gs, n)
    want, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = k * 2.0 ** -24 * mag + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23) * np.abs(want)
    assert np.all(np.abs(_out(y) - want) <= tol)


@pytest.mark.parametrize("m,n,k", [(1, 4112, 320), (2, 5000, 192), (9, 5008, 192), (20, 5008, 208), (2, 16400, 64),
                                   (1, 16401, 576), (30, 16400, 128), (12, 16400, 80), (16, 16401, 64), (2, 16400, 48),
                                   (50, 300, 1024), (31, 4097, 272), (3, 300, 2064), (4, 130, 4096), (5, 520, 2320),
                                   (8, 4096, 2048), (7, 33, 6160), (32, 4200, 1280), (17, 100, 4160), (29, 90, 2192),
                                   (9, 16, 512), (100, 64, 1024), (33, 2048, 528), (1000, 40, 256), (17, 2033, 64)])
def test_exact_on_larger_grids(m, n, k):
    """Row and tile counts on both sides of every choice of launch shape."""
    print(f"[matvec] larger grid {m}x{n}x{k}", flush=True)
    rng = np.random.default_rng(m + n + k)
    x = rng.integers(-8, 9, (m, k)).astype(np.float64)
    q, bs = _grid_matrix(rng, n, k)
    y = fb.nvfp4_matvec(bf16_from_bits(f32_to_bf16(x.astype(np.float32))), torch.from_numpy(q).cuda(),
                        torch.from_numpy(bs).cuda(), torch.ones(1, device="cuda"), out_dtype=torch.float32)
    assert np.array_equal(_out(y), x @ moe.nvfp4_matrix(q, bs, [1.0], n).T)


def test_stacked_tensor_scales_and_every_code():
    """Each run of rows_per_tensor rows has its own scale; every code byte under every e4m3 scale byte but NaN."""
    q = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, axis=1)             # k = 32
    bs = np.stack([np.arange(256) % 127, (np.arange(256) * 3 + 128) % 255], 1).astype(np.uint8)
    bs[(bs & 0x7F) == 0x7F] = 0x38
    gs = np.array([1.0, 0.5, 4.0, 2.0 ** -10], np.float32)
    x = np.zeros((2, 32))
    x[0, [0, 17]] = 1.0                         # single elements, so that sums are exact
    x[1, [1, 30]] = -2.0
    xb = f32_to_bf16(x.astype(np.float32))
    y = fb.nvfp4_matvec(bf16_from_bits(xb), torch.from_numpy(q).cuda(), torch.from_numpy(bs).cuda(),
                        torch.from_numpy(gs).cuda(), rows_per_tensor=64, out_dtype=torch.float32)
    w = moe.nvfp4_matrix(q, bs, gs, 64)
    assert np.array_equal(_out(y), (x @ w.T).astype(np.float32).astype(np.float64))


def test_codes_at_an_eight_byte_offset():
    """Code and scale buffers at the smallest alignment the call allows."""
    rng = np.random.default_rng(5)
    n, k = 40, 512
    q, bs = _grid_matrix(rng, n, k)
    x = rng.integers(-8, 9, (3, k)).astype(np.float64)
    qb = torch.zeros(n * k // 2 + 8, dtype=torch.uint8, device="cuda")
    sb = torch.zeros(n * k // 16 + 1, dtype=torch.uint8, device="cuda")
    qt, st = qb[8:].view(n, k // 2), sb[1:].view(n, k // 16)
    qt.copy_(torch.from_numpy(q))
    st.copy_(torch.from_numpy(bs))
    y = fb.nvfp4_matvec(bf16_from_bits(f32_to_bf16(x.astype(np.float32))), qt, st, torch.ones(1, device="cuda"),
                        out_dtype=torch.float32)
    assert np.array_equal(_out(y), x @ moe.nvfp4_matrix(q, bs, [1.0], n).T)


GROUPS = [([3, 0, 2, 1], 96, 512), ([0, 0, 0], 16, 64), ([1] * 9, 33, 128), ([40, 1, 0, 17], 48, 272),
          ([0, 5], 64, 2048), ([8], 20, 1024), ([0] * 30 + [2] + [0] * 40 + [1], 24, 96),
          # large grids: at most two rows on average (with a group of many among them), some, many; odd k
          ([1, 2, 0, 1, 20, 1, 1, 0, 3, 1, 2, 1, 2, 1, 0, 2] * 2, 560, 192), ([1] * 40, 420, 1088),
          ([5, 1, 17, 0, 8], 4000, 128), ([33, 1, 40, 0, 21], 4000, 64), ([2, 1, 1, 2], 4400, 80),
          ([0] * 300 + [1, 2, 3] + [0] * 300, 6000, 64), ([1] * 1024, 16, 32)]


@pytest.mark.parametrize("sizes,n,k", GROUPS)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("tail", [0, 3])
def test_grouped_exact_on_a_grid(sizes, n, k, gather, tail):
    """Rows behind the last group stay as they were."""
    print(f"[grouped matvec] {len(sizes)} groups of {sum(sizes)} rows, {n}x{k} gather={gather} tail={tail}", flush=True)
    rng = np.random.default_rng(sum(sizes) + n + k)
    g, total = len(sizes), sum(sizes) + tail
    xr = 11 if gather else total
    if total == 0:
        xr = 11
    x = rng.integers(-8, 9, (xr, k)).astype(np.float64)
    mats, qs, ss = [], [], []
    gs = np.exp2(rng.integers(-3, 3, g * 2)).astype(np.float32)
    rpt = n // 2 if n % 2 == 0 else n
    if rpt == n:
        gs = gs[:g]
    for i in range(g):
        q, bs = _grid_matrix(rng, n, k)
        qs.append(q)
        ss.append(bs)
        per = n // rpt
        mats.append(moe.nvfp4_matrix(q, bs, gs[i * per:(i + 1) * per], rpt))
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    ri = rng.integers(0, xr, total).astype(np.int32) if gather else None
    y = torch.full((total, n), 123.0, dtype=torch.float32, device="cuda")
    xt = bf16_from_bits(f32_to_bf16(x.astype(np.float32)))
    if not gather and total == 0:
        xt = xt[:0]
    fb.fp8_nvfp4_grouped_matvec(xt, None if ri is None else torch.from_numpy(ri).cuda(),
                                torch.from_numpy(np.stack(qs)).cuda(), torch.from_numpy(np.stack(ss)).cuda(),
                                torch.from_numpy(gs).cuda(), rpt, torch.from_numpy(off).cuda(), y)
    want, _ = moe.grouped_matvec(x, ri, mats, off, total)
    want = np.where(np.isnan(want), 123.0, want)
    assert np.array_equal(_out(y), want)


def test_grouped_offsets_and_indices_out_of_range_are_clamped():
    """Offsets and indices that break the contract reach nothing outside the buffers; rows whose group and index are
    in range are right."""
    rng = np.random.default_rng(8)
    n, k, g = 32, 128, 4
    x = rng.integers(-8, 9, (3, k)).astype(np.float64)
    q, bs = _grid_matrix(rng, g * n, k)
    ri = np.array([0, 2, 1, -7, 1 << 30, 2], dtype=np.int32)
    off = np.array([-5, 2, 1, 3, 900], dtype=np.int32)
    y = torch.zeros((6, n), dtype=torch.float32, device="cuda")
    fb.fp8_nvfp4_grouped_matvec(bf16_from_bits(f32_to_bf16(x.astype(np.float32))), torch.from_numpy(ri).cuda(),
                                torch.from_numpy(q.reshape(g, n, -1)).cuda(),
                                torch.from_numpy(bs.reshape(g, n, -1)).cuda(), torch.ones(g, device="cuda"), n,
                                torch.from_numpy(off).cuda(), y)
    w = moe.nvfp4_matrix(q, bs, np.ones(1, np.float32), g * n).reshape(g, n, k)
    got = _out(y)
    assert np.array_equal(got[0], x[0] @ w[0].T)                       # group 0: rows [0, 2) after clamping
    assert np.array_equal(got[3:6], np.stack([x[i] @ w[3].T for i in (0, 2, 2)]))


def test_weights_beyond_32_bit_offsets():
    """The last expert of a stack of more than 2^32 bytes of codes."""
    n, k, g = 4096, 7168, 300
    q = torch.zeros((g, n, k // 2), dtype=torch.uint8, device="cuda")
    bs = torch.full((g, n, k // 16), 0x38, dtype=torch.uint8, device="cuda")
    assert q.numel() > 1 << 32
    rng = np.random.default_rng(10)
    qn, bn = _grid_matrix(rng, n, k)
    q[-1].copy_(torch.from_numpy(qn))
    bs[-1].copy_(torch.from_numpy(bn))
    x = rng.integers(-1, 2, (2, k)).astype(np.float64)
    off = torch.zeros(g + 1, dtype=torch.int32, device="cuda")
    off[-1] = 2
    y = fb.nvfp4_grouped_matvec(bf16_from_bits(f32_to_bf16(x.astype(np.float32))), q, bs, torch.ones(g, device="cuda"),
                                off, out_dtype=torch.float32)
    assert np.array_equal(_out(y), x @ moe.nvfp4_matrix(qn, bn, [1.0], n).T)


@pytest.mark.parametrize("sizes", [[2, 1, 0, 2] * 10, [0, 9, 1, 2] * 10, [30, 10, 17, 5] * 10, [7] * 40])
def test_a_large_call_is_its_small_ones(sizes):
    """Weights past the size of the last cache (nontemporal) against the same groups one by one, in exact sums."""
    n, k = 4096, 4096
    g = torch.Generator("cuda").manual_seed(sum(sizes))
    q = torch.randint(0, 256, (len(sizes), n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    bs = torch.full((len(sizes), n, k // 16), 0x38, dtype=torch.uint8, device="cuda")
    gs = torch.full((len(sizes),), 0.5, device="cuda")
    x = torch.randint(-8, 9, (sum(sizes), k), device="cuda", generator=g).to(torch.bfloat16)
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        y = fb.nvfp4_grouped_matvec(x, q, bs, gs, off, out_dtype=dtype)
        at = 0
        for e, rows in enumerate(sizes):
            one = fb.nvfp4_matvec(x[at:at + rows], q[e], bs[e], gs[e:e + 1], out_dtype=dtype)
            assert torch.equal(y[at:at + rows], one), (e, rows)
            at += rows


@pytest.mark.parametrize("m", [1, 2, 5, 20])
def test_a_large_matrix_is_its_rows(m):
    n, k = 80000, 7168
    g = torch.Generator("cuda").manual_seed(m)
    q = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    bs = torch.full((n, k // 16), 0x38, dtype=torch.uint8, device="cuda")
    gs = torch.full((1,), 0.5, device="cuda")
    x = torch.randint(-8, 9, (m, k), device="cuda", generator=g).to(torch.bfloat16)
    y = fb.nvfp4_matvec(x, q, bs, gs, out_dtype=torch.float32)
    for j in range(0, n, 10000):
        one = fb.nvfp4_matvec(x, q[j:j + 10000], bs[j:j + 10000], gs, out_dtype=torch.float32)
        assert torch.equal(y[:, j:j + 10000], one)


@pytest.mark.parametrize("k", [64, 48])
def test_rows_up_to_the_largest_count(k):
    """The last rows of the largest call, more of them than one pass takes: the pass after the last one would begin
    past 2^31.  Rows before the group are left as they were."""
    print(f"[grouped matvec] rows up to 2^31 - 2, k {k}", flush=True)
    total, rows = (1 << 31) - 1, 37
    rng = np.random.default_rng(k)
    x = rng.integers(-8, 9, (5, k)).astype(np.float64)
    q, bs = _grid_matrix(rng, 1, k)
    ri = torch.zeros(total, dtype=torch.int32, device="cuda")
    tail = rng.integers(0, 5, rows)
    ri[-rows:] = torch.from_numpy(tail.astype(np.int32)).cuda()
    off = torch.tensor([total - rows, total], dtype=torch.int32, device="cuda")
    y = torch.full((total, 1), 9.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8_nvfp4_grouped_matvec(bf16_from_bits(f32_to_bf16(x.astype(np.float32))), ri, torch.from_numpy(q[None]).cuda(),
                                torch.from_numpy(bs[None]).cuda(), torch.ones(1, device="cuda"), 1, off, y)
    want = x[tail] @ moe.nvfp4_matrix(q, bs, [1.0], 1).T
    assert np.array_equal(_out(y[-rows:]), _bf16(want))
    assert torch.all(y[:-rows] == 9.0)


# Both ways to multiply (dot products for one or two rows on large grids, the matrix cores otherwise) on values of
# the whole range.  An e2m1 code times the power of two of its scale is exact, and so is its product with x; the
# scale's mantissa, the additions, the tensor scale and fp32 results below the normal range (half of 2^-149 for
# each of the K / 16 blocks' sums and K products) round.
def _range_check(x, q, bs, gs, y, what, nan_rows=()):
    w = moe.nvfp4_matrix(q, bs, gs, len(q))
    ok = np.ones(len(q), bool)
    ok[list(nan_rows)] = False
    want, mag = x @ w[ok].T, np.abs(x) @ np.abs(w[ok]).T
    assert mag.max() < 3.4e38, "the case itself leaves the fp32 range"
    k = x.shape[1]
    got = _out(y)
    tol = (k + k // 16) * 2.0 ** -24 * mag + 2.0 ** -23 * np.abs(want) + 2 * k * 2.0 ** -149 * float(gs[0])
    bad = np.argwhere(~(np.abs(got[:, ok] - want) <= tol + 2.0 ** -149))
    assert len(bad) == 0, (what, len(bad), bad[0], got[:, ok][tuple(bad[0])], want[tuple(bad[0])])
    assert np.all(np.isnan(got[:, ~ok])), what


def _range_case(rng, kind, m, n, k):
    """x [m, k] as bf16 bits, codes and scale bytes of every value but NaN, but as large x allows."""
    q = rng.integers(0, 256, (n, k // 2)).astype(np.uint8)
    bs = rng.integers(0, 256, (n, k // 16)).astype(np.uint8)
    bs[(bs & 0x7F) == 0x7F] = 0x80                       # zeros, of either sign, among them
    bs[rng.random(bs.shape) < 0.1] = 0
    x = rng.standard_normal((m, k))
    if kind == "large":                                  # a few elements near the largest value, under small scales
        at = rng.permutation(k // 16)[:2] * 16 + rng.integers(0, 16, 2)
        x[:, at] = rng.choice([-1, 1], (m, 2)) * np.array([3.3e38, 2e37])
        small = rng.integers(0, 0x11, (n, 2)) | rng.choice([0, 0x80], (n, 2))       # up to 2^-5
        small[rng.random(small.shape) < 0.3] = 0
        bs[:, at // 16] = small
    elif kind == "small":
        x *= 2.0 ** -124
    return f32_to_bf16(x.astype(np.float32)), q, bs


@pytest.mark.parametrize("kind", ["usual", "large", "small"])
@pytest.mark.parametrize("m", [1, 2, 3, 20])
@pytest.mark.parametrize("n,k", [(16400, 192), (16416, 1088), (300, 2064)])
def test_values_of_the_whole_range(kind, m, n, k):
    print(f"[matvec] {kind} values, {m}x{n}x{k}", flush=True)
    rng = np.random.default_rng(m + n)
    xb, q, bs = _range_case(rng, kind, m, n, k)
    gs = np.array([0.37], np.float32)
    y = fb.nvfp4_matvec(bf16_from_bits(xb), torch.from_numpy(q).cuda(), torch.from_numpy(bs).cuda(),
                        torch.from_numpy(gs).cuda(), out_dtype=torch.float32)
    _range_check(bf16_to_f32(xb).astype(np.float64), q, bs, gs, y, kind)


@pytest.mark.parametrize("kind", ["usual", "large", "small"])
def test_grouped_values_of_the_whole_range(kind):
    """Groups of up to two rows and larger ones in one call of a large grid."""
    sizes, n, k = [1, 2, 0, 1, 5, 1, 1, 0, 2, 1, 2, 1, 2, 1, 0, 2] * 2, 600, 320
    rng = np.random.default_rng(12)
    case = [_range_case(rng, kind, s, n, k) for s in sizes]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    gs = np.full(len(sizes), 0.37, np.float32)
    y = fb.nvfp4_grouped_matvec(bf16_from_bits(np.concatenate([c[0] for c in case])),
                                torch.from_numpy(np.stack([c[1] for c in case])).cuda(),
                                torch.from_numpy(np.stack([c[2] for c in case])).cuda(), torch.from_numpy(gs).cuda(),
                                torch.from_numpy(off).cuda(), out_dtype=torch.float32)
    for g, (xb, q, bs) in enumerate(case):
        if sizes[g]:
            _range_check(bf16_to_f32(xb).astype(np.float64), q, bs, gs[:1], y[off[g]:off[g + 1]], (kind, g))


@pytest.mark.parametrize("m,n,k", [(1, 16400, 192), (2, 16400, 192), (5, 16400, 192), (1, 40, 192), (3, 40, 208)])
def test_a_scale_byte_that_is_nan(m, n, k):
    """Its products are NaN, whatever the codes and x; the other matrix rows are as they would be."""
    rng = np.random.default_rng(m + n)
    xb, q, bs = _range_case(rng, "usual", m, n, k)
    q[[3, n - 1]] = 0                                    # codes of 0
    bs[3, 0], bs[17, k // 16 - 1], bs[n - 1, 5] = 0x7F, 0xFF, 0x7F
    gs = np.ones(1, np.float32)
    y = fb.nvfp4_matvec(bf16_from_bits(xb), torch.from_numpy(q).cuda(), torch.from_numpy(bs).cuda(),
                        torch.from_numpy(gs).cuda(), out_dtype=torch.float32)
    _range_check(bf16_to_f32(xb).astype(np.float64), q, bs, gs, y, "NaN scale", nan_rows=(3, 17, n - 1))
