"""Offsets that do not increase: which groups are computed, and that no two of them share rows."""
import pytest
import torch

import fine_grained_moe_gemm_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _groups(off, rows):
    """The rows of each group: nothing where the offsets decrease, leave the buffer, or start before an earlier
    group's end."""
    end, spans = 0, []
    for a, b in zip(off[:-1], off[1:]):
        ok = end <= a <= b <= rows
        spans.append((a, b) if ok else (0, 0))
        end = b if ok else end
    return spans


R = 600
CASES = [[0, R, 0, R], [0, R, 0, R, 0, R] * 40, [0, 100, 50, 120, R], [0, R + 1, 20, 30, R], [30, 10, 40, 20, 50, R],
         [-4, 5, 300, 299, 300, R], [0, 2 ** 31 - 1, -2 ** 31, 100, R], [R, 0, R], [0, R, 0] + [R] * 900,
         [5 * i for i in range(100)] + [3] + [495 + i // 8 for i in range(800)]]


def _check(got, ref, mag, terms):
    assert bool(((got.double() - ref).abs() <= (terms + 2) * 2.0 ** -23 * mag).all())


@pytest.mark.parametrize("n,k", [(8, 64), (520, 136), (72, 4104), (1544, 2056)])
@pytest.mark.parametrize("off", CASES, ids=range(len(CASES)))
def test_groups_never_share_rows(off, n, k):
    gen = torch.Generator(device=DEV).manual_seed(n)
    G, spans = len(off) - 1, _groups(off, R)
    if G * n * k > 1 << 28:
        n, k = 136, 200
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV).to(BF)
    x, w, dy = rand(R, k), rand(G, n, k), rand(R, n)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    y, y8 = torch.full((R, n), 7.0, device=DEV), torch.full((R, n), 7.0, device=DEV)
    dx, dw = torch.full((R, k), 7.0, device=DEV), torch.full((G, n, k), 7.0, device=DEV)
    k8 = k // 16 * 16
    q = torch.randint(-127, 128, (R, k8), generator=gen, device=DEV, dtype=torch.int32).to(torch.int8)
    w8 = torch.randint(-127, 128, (G, n, k8), generator=gen, device=DEV, dtype=torch.int32).to(torch.int8)
    one, ones = torch.ones(R, device=DEV), torch.ones((G, n), device=DEV)
    for call in (lambda: moe.moe_grouped_mm(x, w, o, y), lambda: moe.moe_grouped_mm(dy, w, o, dx, transpose_w=True),
                 lambda: moe.moe_grouped_wgrad(dy, x, o, dw), lambda: moe.moe_grouped_mm_int8(q, one, w8, ones, o, y8)):
        call()
        assert moe.device_error() == moe.MOE_DEVERR_BAD_ROWS
    covered = torch.zeros(R, dtype=torch.bool, device=DEV)
    empty = torch.ones(G, dtype=torch.bool, device=DEV)
    for g, (a, b) in enumerate(spans):
        if a == b:
            continue
        covered[a:b] = True
        empty[g] = False
        xs, ds, wg = x[a:b].double(), dy[a:b].double(), w[g].double()
        _check(y[a:b], xs @ wg.t(), xs.abs() @ wg.abs().t(), k)
        _check(dx[a:b], ds @ wg, ds.abs() @ wg.abs(), n)
        _check(dw[g], ds.t() @ xs, ds.abs().t() @ xs.abs(), b - a)
        ref = q[a:b].double() @ w8[g].double().t()
        assert bool(((y8[a:b].double() - ref).abs() <= 3.01 * 2.0 ** -24 * ref.abs()).all())
    assert bool((dw[empty] == 0).all())
    for t in (y, dx, y8):
        assert bool((t[~covered] == 7.0).all())
