"""The products by group on small integers: every sum is below 2^24, so fp32 holds it exactly in any order and the
result has to be equal, with no tolerance that a lost block, a lost row or a lost share of a sum could hide in.
16-bit results are that integer rounded once, to nearest even."""
import pytest
import torch

import fine_grained_moe_gemm_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FH, FS = torch.bfloat16, torch.float16, torch.float32

RAGGED = [0, 1, 0, 15, 16, 17, 33, 0, 64, 65, 255, 256, 257, 0, 530, 0]
MANY = [0, 1, 17, 32, 33, 64, 0, 100, 129, 160, 200, 224, 225, 256, 257, 300] * 3


def _ints(gen, shape, dtype, most=2):
    return torch.randint(-most, most + 1, shape, generator=gen, device=DEV, dtype=torch.int8).to(dtype)


def _operand(gen, first, rows, spare, width, dtype, strided):
    """`rows` rows of integers between rows of NaN, the columns of a wider buffer of NaN when strided."""
    buf = torch.full((first + rows + spare, width + (24 if strided else 0)), float("nan"), dtype=dtype, device=DEV)
    view = buf[:, 8:8 + width] if strided else buf
    view[first:first + rows] = _ints(gen, (rows, width), dtype)
    return view


def _offsets(sizes, first):
    off = [first]
    for m in sizes:
        off.append(off[-1] + m)
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def _mm(sizes, n, k, dtype, out, transpose, strided=False, accumulate=False):
    gen = torch.Generator(device=DEV).manual_seed(n + k)
    first, spare, rows = 3, 70, sum(sizes)
    x = _operand(gen, first, rows, spare, k, dtype, strided)
    w = _ints(gen, (len(sizes), k, n) if transpose else (len(sizes), n, k), dtype)
    old = _ints(gen, (first + rows + spare, n), out, 100)
    wide = torch.full((old.shape[0], n + 24), float("nan"), dtype=out, device=DEV)
    y = wide[:, 16:16 + n] if strided else old.clone()
    y.copy_(old)
    moe.moe_grouped_mm(x, w, _offsets(sizes, first), y, transpose_w=transpose, accumulate=accumulate)
    assert moe.device_error() == 0
    want, a = old.clone(), first
    for g, m in enumerate(sizes):
        ref = x[a:a + m].double() @ (w[g].double() if transpose else w[g].double().t())
        if accumulate:
            ref = ref + old[a:a + m].double()
        want[a:a + m] = ref.float().to(out)
        a += m
    assert torch.equal(y, want)
    if strided:
        assert bool(wide[:, :16].isnan().all()) and bool(wide[:, 16 + n:].isnan().all())


def _wgrad(sizes, n, k, dtype, out, strided=False, accumulate=False):
    gen = torch.Generator(device=DEV).manual_seed(n + k)
    first, spare, rows = 3, 70, sum(sizes)
    dy, x = (_operand(gen, first, rows, spare, width, dtype, strided) for width in (n, k))
    old = _ints(gen, (len(sizes), n, k), out, 100)
    dw = old.clone()
    moe.moe_grouped_wgrad(dy, x, _offsets(sizes, first), dw, accumulate=accumulate)
    assert moe.device_error() == 0
    a = first
    for g, m in enumerate(sizes):
        ref = dy[a:a + m].double().t() @ x[a:a + m].double()
        if accumulate:
            ref = ref + old[g].double()
        assert torch.equal(dw[g], ref.float().to(out)), f"group {g} of {m} rows"
        a += m


TYPES = [(BF, BF, False), (BF, FS, True), (FH, FH, True), (FH, FS, False)]


@pytest.mark.parametrize("rows,types", [(1, 0), (16, 1), (17, 2), (33, 3), (65, 1), (129, 0), (300, 2)])
@pytest.mark.parametrize("n,k", [(8, 8), (136, 2056), (264, 18432), (16, 65536)])
@pytest.mark.parametrize("transpose", [False, True])
def test_few_rows_over_a_long_axis(rows, types, n, k, transpose):
    dtype, out, accumulate = TYPES[types]
    _mm([rows], n, k, dtype, out, transpose, strided=rows % 2 == 1, accumulate=accumulate)


@pytest.mark.parametrize("dtype,out,accumulate", TYPES)
@pytest.mark.parametrize("sizes", [[222], [256], [129, 0, 3], [513], [70, 71]])
@pytest.mark.parametrize("n,k", [(1544, 4104), (392, 18432)])
@pytest.mark.parametrize("transpose", [False, True])
def test_few_wide_tiles_over_a_long_axis(sizes, n, k, transpose, dtype, out, accumulate):
    _mm(sizes, n, k, dtype, out, transpose, strided=len(sizes) > 1, accumulate=accumulate)


@pytest.mark.parametrize("dtype,out,accumulate", TYPES)
@pytest.mark.parametrize("sizes,n,k", [(RAGGED, 152, 328), (RAGGED, 1048, 1160), (MANY, 4104, 72), (MANY, 4104, 136),
                                       ([9480], 2056, 8200), ([5000, 4480], 2056, 1048)])
@pytest.mark.parametrize("transpose", [False, True])
def test_products(sizes, n, k, transpose, dtype, out, accumulate):
    _mm(sizes, n, k, dtype, out, transpose, strided=True, accumulate=accumulate)


@pytest.mark.parametrize("rows,types", [(1, 0), (15, 1), (16, 2), (63, 3), (65, 0), (257, 1), (1000, 2), (4099, 3)])
@pytest.mark.parametrize("n,k", [(8, 8), (72, 136), (136, 264)])
def test_gradients_of_few_tiles(rows, types, n, k):
    dtype, out, accumulate = TYPES[types]
    _wgrad([rows], n, k, dtype, out, accumulate=accumulate)


@pytest.mark.parametrize("dtype,out,accumulate", TYPES)
@pytest.mark.parametrize("sizes", [[20011], [16384], [9000, 0, 30, 5000], [0, 12345]])
@pytest.mark.parametrize("n,k", [(552, 488), (264, 1032), (1000, 256)])
def test_gradients_of_few_wide_tiles_over_many_rows(sizes, n, k, dtype, out, accumulate):
    _wgrad(sizes, n, k, dtype, out, strided=True, accumulate=accumulate)


@pytest.mark.parametrize("dtype,out,accumulate", TYPES)
@pytest.mark.parametrize("sizes,n,k", [(RAGGED, 152, 328), (RAGGED, 1048, 1160), ([700, 3, 1500, 513, 0, 1] * 20, 264, 328),
                                       ([20000, 100, 0, 8200, 9000] + [0] * 300, 264, 328), ([70001] + [0] * 300, 136, 264)])
def test_gradients(sizes, n, k, dtype, out, accumulate):
    _wgrad(sizes, n, k, dtype, out, strided=True, accumulate=accumulate)
