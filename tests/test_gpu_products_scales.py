"""Scales of the 8-bit products over the whole range of fp32: a product of the two that leaves the normal numbers
must not reach the result.

Tolerance: the conversion of the sum and two products are three roundings of 2^-24 each; below the normal numbers one
of them is half a step of 2^-149 instead."""
import pytest
import torch

import fine_grained_moe_gemm_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"

RAGGED = [0, 1, 15, 17, 33, 64, 65, 255, 257, 0, 300]
MANY = [0, 1, 17, 32, 33, 64, 0, 100, 129, 160, 200, 224, 225, 256, 257, 300] * 3
# rows: ordinary, near and below the smallest normal number, large, the largest that moe_quantize_int8 writes
ROWS = [1.3e-3, 2.0 ** -126 * 1.37, 2.0 ** -140 * 1.9, 2.0 ** -149, 1.7, 2.0 ** 96 * 1.1, 2.0 ** 100 * 1.3, 2.0 ** 121 * 1.01]
COLUMNS = [1.1e-3, 2.0 ** -10 * 1.7, 2.0 ** -60 * 1.2, 2.0 ** -130 * 1.5, 2.0 ** -149 * 3, 2.0 ** 60 * 1.6, 2.0 ** 101 * 1.4, 1.9]


@pytest.mark.parametrize("ordinary_rows", [False, True])
@pytest.mark.parametrize("sizes,n,k", [
    (RAGGED, 1032, 208),      # tiles of pairs
    (RAGGED, 1032, 8208),
    (MANY, 4104, 128),        # the epilogue's halves take tiles in turn
    ([16], 136, 18432),       # CTAs share a sum
    ([250], 1032, 8208),      # pairs share a sum
    ([3], 8, 16),
])
def test_scales_of_every_size(sizes, n, k, ordinary_rows):
    gen = torch.Generator(device=DEV).manual_seed(n + k)
    rows, groups = sum(sizes), len(sizes)
    code = lambda shape: torch.randint(-128, 128, shape, generator=gen, device=DEV, dtype=torch.int32).to(torch.int8)
    q, w = code((rows, k)), code((groups, n, k))
    q[::5] = 0                                             # sums of zero under every scale
    pick = lambda v, shape: torch.tensor(v, device=DEV)[torch.randint(len(v), shape, generator=gen, device=DEV)]
    sx, sw = pick(ROWS[:5] if ordinary_rows else ROWS, (rows,)), pick(COLUMNS, (groups, n))
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    y = torch.full((rows, n), 7.0, device=DEV)
    moe.moe_grouped_mm_int8(q, sx, w, sw, off, y)
    assert moe.device_error() == 0
    a = 0
    for g, m in enumerate(sizes):
        ref = (q[a:a + m].double() @ w[g].double().t()) * (sx[a:a + m].double()[:, None] * sw[g].double())
        got = y[a:a + m].double()
        over = ref.abs() >= 2.0 ** 128                     # no value here lies within a rounding of it
        assert bool((got[over] == ref[over].sign() * float("inf")).all())
        bad = ~over & ~((got - ref).abs() <= 3.01 * 2.0 ** -24 * ref.abs() + 2.0 ** -149)
        assert not bool(bad.any()), (g, m, int(bad.sum()), got[bad][:4].tolist(), ref[bad][:4].tolist())
        a += m


@pytest.mark.parametrize("sizes,n,k", [(RAGGED, 1032, 208), (MANY, 4104, 128), ([16], 136, 18432), ([250], 1032, 8208)])
def test_scales_that_are_not_finite(sizes, n, k):
    """A row or a channel whose scale is infinite or no number has no finite result where its sum is zero (the codes
    of a row with an infinity are zeros); its neighbours are not touched."""
    gen = torch.Generator(device=DEV).manual_seed(k)
    rows, groups = sum(sizes), len(sizes)
    code = lambda shape: torch.randint(-127, 128, shape, generator=gen, device=DEV, dtype=torch.int32).to(torch.int8)
    q, w = code((rows, k)), code((groups, n, k))
    sx, sw = torch.rand(rows, generator=gen, device=DEV) + 0.5, torch.rand((groups, n), generator=gen, device=DEV) + 0.5
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    clean = torch.empty((rows, n), device=DEV)
    moe.moe_grouped_mm_int8(q, sx, w, sw, off, clean)
    bad_rows, bad_columns = [rows // 3, rows - 1], [5, n - 2]
    q2, sx2, sw2 = q.clone(), sx.clone(), sw.clone()
    q2[bad_rows] = 0
    sx2[bad_rows[0]], sx2[bad_rows[1]] = float("inf"), float("nan")
    sw2[:, bad_columns[0]], sw2[:, bad_columns[1]] = float("nan"), float("inf")
    y = torch.empty((rows, n), device=DEV)
    moe.moe_grouped_mm_int8(q2, sx2, w, sw2, off, y)
    assert moe.device_error() == 0
    assert bool(y[bad_rows].isnan().all())
    assert bool(y[:, bad_columns[0]].isnan().all()) and not bool(y[:, bad_columns[1]].isfinite().any())
    keep_r, keep_c = torch.ones(rows, dtype=torch.bool, device=DEV), torch.ones(n, dtype=torch.bool, device=DEV)
    keep_r[bad_rows], keep_c[bad_columns] = False, False
    # the two orders of the scales round differently: three roundings each
    got, want = y[keep_r][:, keep_c], clean[keep_r][:, keep_c]
    assert bool(((got - want).abs() <= 6.01 * 2.0 ** -24 * want.abs()).all())
