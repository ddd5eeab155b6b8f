"""The products grouped by expert, SwiGLU with its gradient and the int8 codes on a B200, against plain 64-bit
arithmetic.

Tolerances.  Products of two 16-bit values are exact in fp32; a sum of m terms in fp32 with additions off by at
most one unit of 2^-23 of the running magnitude is off by at most m 2^-23 sum |x w| (_sum_bound).  A result in a
type t is then off by half a step more, eps(t) / 2 of its value (fp32 results: that is inside the sum's bound).
Integer sums are exact; the fp32 conversion and the two scales are three roundings."""
import numpy as np
import pytest
import torch

import fine_grained_moe_gemm_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FH, FS = torch.bfloat16, torch.float16, torch.float32

# rows of the groups: empty ones, one row, around 16, 32, 64 and 256, several chunks
RAGGED = [0, 1, 0, 15, 16, 17, 33, 0, 64, 65, 255, 256, 257, 0, 530, 0]
FEW = [3, 0, 1, 7]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rand(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _wide(t, pad=24):
    """The same matrix as a slice of a wider buffer whose other values are NaN."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
    v = buf[:, 8:8 + t.shape[1]]
    v.copy_(t)
    return v


def _offsets(sizes, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(sizes)]), dtype=torch.int32, device=DEV)


def _eps(dtype):
    return torch.finfo(dtype).eps / 2


def _within(got, ref, bound, what="result"):
    got = got.double()
    bad = ~((got - ref).abs() <= bound)
    if bool(bad.any()):
        worst = float((got - ref).abs().nan_to_num(1e30).max())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst error {worst}, first at "
                             f"{bad.nonzero()[0].tolist()}")


def _mm_ref(x, w, sizes, first, transpose):
    """Reference and its sum of magnitudes, rows of the groups only."""
    ref, mag, a = [], [], first
    for g, m in enumerate(sizes):
        xs, ws = x[a:a + m].double(), w[g].double() if transpose else w[g].double().t()
        ref.append(xs @ ws)
        mag.append(xs.abs() @ ws.abs())
        a += m
    return torch.cat(ref), torch.cat(mag)


def _mm_case(sizes, n, k, dtype, out, transpose, seed=0, first=0, spare=0, strided=False, accumulate=False):
    gen = _gen(seed)
    rows, end = first + sum(sizes) + spare, first + sum(sizes)
    x = _rand(gen, (rows, k), dtype)
    x[:first] = float("nan")           # rows outside the groups must not matter
    x[end:] = float("nan")
    w = _rand(gen, (len(sizes), k, n) if transpose else (len(sizes), n, k), dtype, 0.1)
    old = _rand(gen, (rows, n), out)
    y = _wide(old) if strided else old.clone()
    if strided:
        x = _wide(x)
    moe.moe_grouped_mm(x, w, _offsets(sizes, first), y, transpose_w=transpose, accumulate=accumulate)
    torch.cuda.synchronize()
    assert moe.device_error() == 0
    ref, mag = _mm_ref(x, w, sizes, first, transpose)
    bound = (k + 2) * 2.0 ** -23 * mag
    if accumulate:
        ref = ref + old[first:end].double()
        bound = bound + 2.0 ** -23 * old[first:end].double().abs()
    if out != FS:
        bound = bound * (1 + _eps(out)) + _eps(out) * ref.abs()
        if out == FH:
            bound = bound + 2.0 ** -25     # half a step of the subnormal numbers
    _within(y[first:end], ref, bound)
    assert torch.equal(y[:first], old[:first]) and torch.equal(y[end:], old[end:])
    if strided:
        whole = y.as_strided((rows, n + 24), (n + 24, 1), 0)
        assert bool(whole[:, :8].isnan().all()) and bool(whole[:, 8 + n:].isnan().all())


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("n,k", [(8, 8), (64, 64), (136, 72), (264, 1160), (512, 256), (1032, 200), (1040, 8)])
@pytest.mark.parametrize("sizes", [FEW, RAGGED])
def test_mm_sizes(sizes, n, k, transpose):
    _mm_case(sizes, n, k, BF, FS, transpose, seed=n + k)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n", [152, 1048])   # few tiles, and enough for every SM
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, FS), (FH, FH), (FH, FS)])
def test_mm_types(dtype, out, n, accumulate, strided, transpose):
    _mm_case(RAGGED, n, 328, dtype, out, transpose, seed=7, first=5, spare=9, strided=strided, accumulate=accumulate)


@pytest.mark.parametrize("sizes", [[1], [5], [300], [0, 0, 0, 1000], [1] * 300, [0] * 1023 + [2], [2049, 0, 1]])
@pytest.mark.parametrize("transpose", [False, True])
def test_mm_groups(sizes, transpose):
    _mm_case(sizes, 256, 128, BF, BF, transpose, seed=len(sizes))


def test_mm_without_offsets_and_without_rows():
    gen = _gen(3)
    x, w = _rand(gen, (77, 96), BF), _rand(gen, (1, 40, 96), BF)
    y = torch.empty((77, 40), dtype=FS, device=DEV)
    moe.moe_grouped_mm(x, w, None, y)
    ref, mag = _mm_ref(x, w, [77], 0, False)
    _within(y, ref, 98 * 2.0 ** -23 * mag)
    moe.moe_grouped_mm(x[:0], w, None, y[:0])
    assert moe.device_error() == 0


def _wgrad_case(sizes, n, k, dtype, out, seed=0, first=0, spare=0, strided=False, accumulate=False, poison=None):
    gen = _gen(seed)
    rows, end = first + sum(sizes) + spare, first + sum(sizes)
    dy, x = _rand(gen, (rows, n), dtype), _rand(gen, (rows, k), dtype)
    for t in (dy, x):
        t[:first] = float("nan")
        t[end:] = float("nan")
    starts = np.concatenate([[first], first + np.cumsum(sizes)])
    if poison is not None:
        dy[starts[poison]:starts[poison + 1]] = float("nan")
        x[starts[poison]:starts[poison + 1]] = float("inf")
    if strided:
        dy, x = _wide(dy), _wide(x)
    old = _rand(gen, (len(sizes), n, k), out)
    dw = old.clone()
    moe.moe_grouped_wgrad(dy, x, _offsets(sizes, first), dw, accumulate=accumulate)
    torch.cuda.synchronize()
    assert moe.device_error() == 0
    for g, m in enumerate(sizes):
        if g == poison:
            assert m == 0 or bool(dw[g].isnan().all())
            continue
        a, b = dy[starts[g]:starts[g + 1]].double(), x[starts[g]:starts[g + 1]].double()
        ref, bound = a.t() @ b, (m + 2) * 2.0 ** -23 * (a.abs().t() @ b.abs())
        if accumulate:
            ref, bound = ref + old[g].double(), bound + 2.0 ** -23 * old[g].double().abs()
        if out != FS:
            bound = bound * (1 + _eps(out)) + _eps(out) * ref.abs() + (2.0 ** -25 if out == FH else 0.0)
        if m == 0:
            assert torch.equal(dw[g], old[g] if accumulate else torch.zeros_like(old[g]))
        _within(dw[g], ref, bound, f"group {g} of {m} rows")


@pytest.mark.parametrize("n,k", [(8, 8), (64, 64), (136, 72), (264, 520), (512, 256), (1032, 200)])
@pytest.mark.parametrize("sizes", [FEW, RAGGED])
def test_wgrad_sizes(sizes, n, k):
    _wgrad_case(sizes, n, k, BF, FS, seed=n + k)


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n", [152, 1048])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, FS), (FH, FH), (FH, FS)])
def test_wgrad_types(dtype, out, n, accumulate, strided):
    _wgrad_case(RAGGED, n, 328, dtype, out, seed=11, first=3, spare=70, strided=strided, accumulate=accumulate)


@pytest.mark.parametrize("n", [136, 1032])
@pytest.mark.parametrize("poison", [3, 9, 11])
def test_wgrad_neighbours_do_not_leak(poison, n):
    """A group of NaN and infinities lies right behind another group's last rows, inside its 64-row block."""
    _wgrad_case(RAGGED, n, 136, BF, FS, seed=12, poison=poison)


@pytest.mark.parametrize("dtype", [BF, FH])
def test_long_fp32_sums_keep_their_precision(dtype):
    """The tensor core cuts its partial sums off; within 512 terms (32 additions) that is at most 32 x 2^-23 of the
    sum and half of it on average, 2e-6; adding the segments in fp32 must not let it grow with the length."""
    gen = _gen(21)
    for m in (512, 513, 4096, 30001):
        dy, x = _rand(gen, (m, 264), dtype), _rand(gen, (m, 136), dtype)
        dw = torch.empty((1, 264, 136), device=DEV)
        moe.moe_grouped_wgrad(dy, x, None, dw)
        ref = dy.double().t() @ x.double()
        assert float((dw[0].double() - ref).norm() / ref.norm()) <= 2e-6, m
    for k in (512, 520, 4096, 18432, 65536):
        for transpose in (False, True):
            x, w = _rand(gen, (300, k), dtype), _rand(gen, (1, k, 136) if transpose else (1, 136, k), dtype)
            y = torch.empty((300, 136), device=DEV)
            moe.moe_grouped_mm(x, w, None, y, transpose_w=transpose)
            ref = x.double() @ (w[0].double() if transpose else w[0].double().t())
            assert float((y.double() - ref).norm() / ref.norm()) <= 2e-6, k
    assert moe.device_error() == 0


@pytest.mark.parametrize("n", [136, 1032])   # few tiles, and enough for every SM
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("strided", [False, True])
def test_long_fp32_sums_ragged(transpose, strided, n):
    _mm_case(RAGGED, n, 1048, BF, FS, transpose, seed=31, first=2, spare=3, strided=strided, accumulate=True)


@pytest.mark.parametrize("n", [136, 1032])
@pytest.mark.parametrize("accumulate", [False, True])
def test_long_fp32_gradients_ragged(accumulate, n):
    _wgrad_case([0, 700, 3, 1500, 0, 512, 513, 1025], n, 264, BF, FS, seed=32, first=1, spare=5, accumulate=accumulate,
                poison=4)
    _wgrad_case([700, 3, 1500], n, 264, FH, FS, seed=33, accumulate=accumulate, poison=1)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 63, 65, 128, 129, 300])
@pytest.mark.parametrize("n,k", [(8, 8), (136, 2056), (264, 18432)])
@pytest.mark.parametrize("transpose", [False, True])
def test_mm_one_group_of_few_rows(rows, n, k, transpose):
    """Few tiles over a long axis: the axis is shared by up to eight CTAs."""
    _mm_case([rows], n, k, BF, BF if rows % 2 else FS, transpose, seed=rows, first=3, spare=2, accumulate=rows % 3 == 0)


@pytest.mark.parametrize("sizes", [[222], [256], [129, 0, 3], [513], [70, 71]])
@pytest.mark.parametrize("n,k", [(1544, 4104), (392, 18432)])
@pytest.mark.parametrize("transpose", [False, True])
def test_mm_few_wide_tiles_over_a_long_axis(sizes, n, k, transpose):
    _mm_case(sizes, n, k, FH, FH if len(sizes) > 1 else FS, transpose, seed=n, first=1, spare=2, accumulate=len(sizes) == 3)


@pytest.mark.parametrize("rows", [1, 15, 16, 63, 64, 65, 257, 1000, 4099])
@pytest.mark.parametrize("n,k", [(8, 8), (72, 136), (136, 264)])
def test_wgrad_one_group_of_few_tiles(rows, n, k):
    _wgrad_case([rows], n, k, FH, FH if rows % 2 else FS, seed=rows, first=1, spare=70, accumulate=rows % 3 == 0)


@pytest.mark.parametrize("sizes", [[20011], [16384], [9000, 0, 30, 5000], [0, 12345]])
@pytest.mark.parametrize("n,k", [(552, 488), (264, 1032), (1000, 256)])
def test_wgrad_few_wide_tiles_of_many_rows(sizes, n, k):
    _wgrad_case(sizes, n, k, BF, BF if len(sizes) == 4 else FS, seed=n, first=2, spare=70, accumulate=len(sizes) == 2,
                poison=2 if len(sizes) == 4 else None)


def test_wgrad_without_rows_is_zero():
    dw = torch.full((3, 16, 24), float("nan"), device=DEV)
    none = torch.empty((0, 16), dtype=BF, device=DEV), torch.empty((0, 24), dtype=BF, device=DEV)
    moe.moe_grouped_wgrad(*none, _offsets([0, 0, 0]), dw)
    assert bool((dw == 0).all())
    dw.fill_(2.0)
    moe.moe_grouped_wgrad(*none, _offsets([0, 0, 0]), dw, accumulate=True)
    assert bool((dw == 2.0).all())


@pytest.mark.parametrize("bad,g_bad", [([0, 5, 3, 3], 1), ([-1, 5, 6, 9], 0), ([0, 5, 6, 11], 2)])
def test_bad_offsets_are_empty_groups(bad, g_bad):
    """One of three groups decreases, starts below zero or ends behind the ten rows; the others are computed."""
    gen = _gen(5)
    off = torch.tensor(bad, dtype=torch.int32, device=DEV)
    x, w = _rand(gen, (10, 32), BF), _rand(gen, (3, 16, 32), BF)
    dy = _rand(gen, (10, 16), BF)
    y = torch.full((10, 16), 7.0, device=DEV)
    dw = torch.full((3, 16, 32), 7.0, device=DEV)
    moe.moe_grouped_mm(x, w, off, y)
    assert moe.device_error() == moe.MOE_DEVERR_BAD_ROWS
    moe.moe_grouped_wgrad(dy, x, off, dw)
    assert moe.device_error() == moe.MOE_DEVERR_BAD_ROWS
    covered = torch.zeros(10, dtype=torch.bool, device=DEV)
    for g in range(3):
        a, b = bad[g], bad[g + 1]
        if g == g_bad:
            assert bool((dw[g] == 0).all())
            continue
        covered[a:b] = True
        xs, ds = x[a:b].double(), dy[a:b].double()
        _within(dw[g], ds.t() @ xs, 12 * 2.0 ** -23 * (ds.abs().t() @ xs.abs()))
        _within(y[a:b], xs @ w[g].double().t(), 34 * 2.0 ** -23 * (xs.abs() @ w[g].double().abs().t()))
    assert bool((y[~covered] == 7.0).all())


# ------------------------------------------------------------------ int8
@pytest.mark.parametrize("dtype", [BF, FH, FS])
@pytest.mark.parametrize("rows,k", [(1, 16), (3, 48), (7, 512), (130, 7168), (2, 18432), (5, 32768), (4000, 80)])
def test_int8_codes(rows, k, dtype):
    gen = _gen(k)
    x = _rand(gen, (rows, k), dtype)
    x[0] = 0.0
    if rows > 2:
        # quotients on the border: x = (c + 1/2) s exactly, with s a power of two
        x[1] = ((torch.arange(k, device=DEV) % 254 - 127).float() + 0.5).clamp(-126.5, 126.5).to(dtype)
        x[1, 0] = 127.0
        x[2] = x[2] * 2.0 ** (-120 if dtype != FH else -14)
    if rows > 4:
        x[3, k // 2] = float("inf")
        x[4, k - 1] = float("nan")
    x = _wide(x) if rows % 2 else x
    q = torch.full((rows, k), 99, dtype=torch.int8, device=DEV)
    sx = torch.full((rows,), -1.0, device=DEV)
    moe.moe_quantize_int8(x, q, sx)
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    if rows > 4:
        bad[3] = bad[4] = True
        assert bool((q[3:5] == 0).all()) and not bool(sx[3:5].isfinite().any())
    # one fp32 product (the product of two fp32 numbers is exact in 64 bits)
    ref_s = (x.double().abs().amax(1) * float(np.float32(1) / np.float32(127))).float()
    ref_s = torch.where(ref_s == 0, torch.ones_like(ref_s), ref_s)
    assert torch.equal(sx[~bad], ref_s[~bad])
    ref_q = torch.round(x.double() / ref_s.double()[:, None]).clamp(-127, 127)
    assert torch.equal(q[~bad].double(), ref_q[~bad])


def test_int8_codes_next_to_the_border():
    """fp32 values one ulp around every border of a scale that is no power of two."""
    s = np.float32(0.1234567)
    amax = np.float32(s * np.float32(127.0))
    s = np.float32(amax * (np.float32(1) / np.float32(127)))
    mid = ((np.arange(-127, 127) + 0.5) * np.float64(s)).astype(np.float32)
    x = np.concatenate([mid, np.nextafter(mid, np.float32(np.inf)), np.nextafter(mid, np.float32(-np.inf))])
    x = np.concatenate([[amax], x, np.zeros((-len(x) - 1) % 16, np.float32)]).astype(np.float32)
    t = torch.from_numpy(x)[None].to(DEV)
    q, sx = torch.empty(t.shape, dtype=torch.int8, device=DEV), torch.empty(1, device=DEV)
    moe.moe_quantize_int8(t, q, sx)
    assert float(sx) == float(s)
    assert np.array_equal(q.cpu().numpy()[0], np.rint(x.astype(np.float64) / np.float64(s)))


def _codes(gen, shape):
    return torch.randint(-128, 128, shape, generator=gen, device=DEV, dtype=torch.int32).to(torch.int8)


@pytest.mark.parametrize("out", [BF, FH, FS])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("sizes,n,k", [(FEW, 8, 16), (RAGGED, 136, 80), (RAGGED, 264, 1168), (RAGGED, 1032, 208), ([16], 1032, 2064),
                                       ([16], 136, 18432), ([250], 1032, 8208), ([100, 90], 392, 16400),
                                       ([300], 256, 128), ([0] * 200 + [1], 64, 32), ([2], 16, 65536)])
def test_mm_int8(sizes, n, k, accumulate, out):
    gen = _gen(n + k)
    first, spare = (0, 0) if len(sizes) == 1 else (4, 6)
    rows, end = first + sum(sizes) + spare, first + sum(sizes)
    q, w = _codes(gen, (rows, k)), _codes(gen, (len(sizes), n, k))
    if sizes == [2]:   # the largest sums: 65536 products of 128 * 128
        q.fill_(-128)
        w.fill_(-128)
    sx = torch.rand(rows, generator=gen, device=DEV) * 1e-3 + 1e-4
    sw = torch.rand((len(sizes), n), generator=gen, device=DEV) * 1e-2 + 1e-3
    old = _rand(gen, (rows, n), out)
    y = old.clone()
    moe.moe_grouped_mm_int8(q, sx, w, sw, _offsets(sizes, first) if len(sizes) > 1 else None, y, accumulate=accumulate)
    assert moe.device_error() == 0
    ref, a = [], first
    for g, m in enumerate(sizes):
        acc = q[a:a + m].double() @ w[g].double().t()
        ref.append(acc * sx[a:a + m].double()[:, None] * sw[g].double())
        a += m
    ref = torch.cat(ref)
    bound = 3.01 * 2.0 ** -24 * ref.abs()
    if accumulate:
        ref, o = ref + old[first:end].double(), old[first:end].double().abs()
        bound = bound + 2.0 ** -24 * (ref.abs() + bound)
    bound = bound * (1 + _eps(out)) + _eps(out) * ref.abs() + (2.0 ** -25 if out == FH else 0.0)
    _within(y[first:end], ref, bound)
    assert torch.equal(y[:first], old[:first]) and torch.equal(y[end:], old[end:])


# many groups over short sums: enough tiles that every pair of SMs takes six or more, of all widths
MANY = [0, 1, 17, 32, 33, 64, 0, 100, 129, 160, 200, 224, 225, 256, 257, 300] * 3


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("k", [8, 64, 72, 128, 136])
@pytest.mark.parametrize("dtype,out,accumulate", [(BF, BF, False), (FH, FH, True), (BF, FS, False), (FH, FS, True)])
def test_mm_many_groups_of_short_sums(dtype, out, accumulate, k, transpose):
    _mm_case(MANY, 4104, k, dtype, out, transpose, seed=k, first=3, spare=5, strided=True, accumulate=accumulate)


@pytest.mark.parametrize("out,accumulate", [(BF, False), (FH, True), (FS, False), (FS, True)])
@pytest.mark.parametrize("k", [16, 112, 128, 240, 256, 272])
def test_mm_int8_many_groups_of_short_sums(k, out, accumulate):
    test_mm_int8(MANY, 4104, k, accumulate, out)


# ------------------------------------------------------------------ SwiGLU
def _swiglu_ref(gate, up, coef, dh=None):
    a, b = gate.double(), up.double()
    c = coef.double()[:, None] if coef is not None else 1.0
    s = torch.sigmoid(a)
    h = c * a * s * b
    if dh is None:
        return h
    d = dh.double()
    return h, c * d * b * s * (1 + a * (1 - s)), c * d * a * s, (d * a * s * b)


def _swiglu_bound(out, size):
    """fp32 steps: the exponential and the quotients are good to 2^-21 (fast forms: |a| 2^-24 in the exponent's
    argument as well, |a| < 16 where the value matters), four more roundings; `size` bounds the terms."""
    return 2.0 ** -18 * size + _eps(out) * size * 1.01 + (2.0 ** -24 if out == FH else 1e-30)


@pytest.mark.parametrize("dtype", [BF, FH, FS])
@pytest.mark.parametrize("rows,width", [(1, 8), (3, 24), (5, 128), (257, 200), (33, 2048), (300, 18432 // 8), (2, 65536)])
@pytest.mark.parametrize("with_coef", [False, True])
def test_swiglu(rows, width, dtype, with_coef):
    gen = _gen(rows + width)
    gate, up, dh = (_rand(gen, (rows, width), dtype, s) for s in (2.0, 1.0, 0.5))
    gate[0, 0], gate[0, 1], gate[0, 2], gate[0, 3] = -100.0, 100.0, 0.0, -20.0
    coef = torch.rand(rows, generator=gen, device=DEV) if with_coef else None
    if rows > 2 and with_coef:
        coef[1] = 0.0
    gate, up = _wide(gate), _wide(up)
    h = torch.empty((rows, width), dtype=dtype, device=DEV)
    dgate, dup = _wide(torch.zeros_like(h)), torch.empty_like(h)
    dcoef = torch.empty(rows, device=DEV) if with_coef else None
    moe.moe_swiglu(gate, up, h, coef=coef)
    moe.moe_swiglu_backward(dh, gate, up, dgate, dup, coef=coef, dcoef=dcoef)
    rh, rg, ru, dots = _swiglu_ref(gate, up, coef, dh)
    _within(h, rh, _swiglu_bound(dtype, rh.abs()))
    a, c = gate.double(), coef.double()[:, None] if with_coef else 1.0
    s = torch.sigmoid(a)
    # the terms s and a s (1 - s) of dgate may cancel: their magnitudes bound the error
    _within(dgate, rg, _swiglu_bound(dtype, rg.abs()) + 2.0 ** -18 * (c * dh.double() * up.double()).abs() * (s + (a * s * (1 - s)).abs()))
    _within(dup, ru, _swiglu_bound(dtype, ru.abs()))
    if with_coef:
        _within(dcoef, dots.sum(1), (2.0 ** -18 + (width + 32) * 2.0 ** -24) * dots.abs().sum(1) + 1e-30)
    # in place: the gradients over gate and up, and over dh
    g2, u2, d2 = gate.clone(), up.clone(), dh.clone()
    moe.moe_swiglu_backward(d2, g2, u2, g2, u2, coef=coef)
    assert torch.equal(g2, dgate) and torch.equal(u2, dup)
    g2 = gate.clone()
    moe.moe_swiglu_backward(d2, g2, up, g2, d2, coef=coef)
    assert torch.equal(g2, dgate) and torch.equal(d2, dup)
    g2 = gate.clone()
    moe.moe_swiglu(g2, up, g2, coef=coef)
    assert torch.equal(g2, h)


def test_swiglu_against_differences():
    gen = _gen(17)
    gate, up, dh = (_rand(gen, (6, 40), FS, s) for s in (1.5, 1.0, 1.0))
    coef = torch.rand(6, generator=gen, device=DEV) + 0.5
    dg, du, dc = torch.empty_like(gate), torch.empty_like(gate), torch.empty_like(coef)
    moe.moe_swiglu_backward(dh, gate, up, dg, du, coef=coef, dcoef=dc)
    step = 2.0 ** -6

    def f(g, u, c):
        h = torch.empty_like(g)
        moe.moe_swiglu(g, u, h, coef=c)
        return h.double() * dh.double()

    # central difference: step^2 / 6 of the third derivative (of SiLU: below 1 everywhere) and the forward's
    # fp32 error (2^-20 of values below 64) over the step
    scale = (dh * coef[:, None]).double().abs()
    tol = (step ** 2 / 6 * up.double().abs() + 2.0 ** -20 * 64 / step) * scale + 1e-6
    _within(dg, (f(gate + step, up, coef) - f(gate - step, up, coef)) / (2 * step), tol)
    _within(du, (f(gate, up + step, coef) - f(gate, up - step, coef)) / (2 * step), 2.0 ** -20 * 64 / step * scale + 1e-6)
    _within(dc, ((f(gate, up, coef + step) - f(gate, up, coef - step)) / (2 * step)).sum(1),
            40 * 2.0 ** -20 * 64 / step * dh.double().abs().amax(1) + 1e-6)


@pytest.mark.parametrize("width", [24, 256, 8192])
def test_coefficient_gradient_in_place(width):
    gen = _gen(width)
    g, u, d = (_rand(gen, (300, width), BF) for _ in range(3))
    c = torch.rand(300, generator=gen, device=DEV)
    dg, du, dc = torch.empty_like(g), torch.empty_like(g), torch.empty_like(c)
    moe.moe_swiglu_backward(d, g, u, dg, du, coef=c, dcoef=dc)
    over = c.clone()
    moe.moe_swiglu_backward(d, g, u, g, u, coef=over, dcoef=over)
    assert torch.equal(over, dc) and torch.equal(g, dg) and torch.equal(u, du)


@pytest.mark.parametrize("count", [0, 1, 5, 12])
def test_rows_behind_the_count_stay(count):
    gen = _gen(count)
    gate, up, dh = (_rand(gen, (12, 64), BF) for _ in range(3))
    n = torch.tensor([0, count], dtype=torch.int32, device=DEV)[1:]
    h, dg, du = (torch.full((12, 64), 3.0, dtype=BF, device=DEV) for _ in range(3))
    dc, coef = torch.full((12,), 3.0, device=DEV), torch.ones(12, device=DEV)
    q, sx = torch.full((12, 64), 3, dtype=torch.int8, device=DEV), torch.full((12,), 3.0, device=DEV)
    moe.moe_swiglu(gate, up, h, coef=coef, n_rows=n)
    moe.moe_swiglu_backward(dh, gate, up, dg, du, coef=coef, dcoef=dc, n_rows=n)
    moe.moe_quantize_int8(gate, q, sx, n_rows=n)
    assert moe.device_error() == 0
    for t in (h, dg, du, dc, q, sx):
        assert bool((t[count:] == 3).all())
    full = torch.empty_like(h)
    moe.moe_swiglu(gate, up, full, coef=coef)
    assert torch.equal(h[:count], full[:count])
    n.fill_(13)
    moe.moe_swiglu(gate, up, h, n_rows=n)
    assert moe.device_error() == moe.MOE_DEVERR_BAD_ROWS


# ------------------------------------------------------------------ together
def _ffn(sizes, d, hid, seed=0):
    gen = _gen(seed)
    G, R = len(sizes), sum(sizes)
    t = {"x": _rand(gen, (R, d), BF), "dy": _rand(gen, (R, d), BF), "off": _offsets(sizes),
         "coef": torch.rand(R, generator=gen, device=DEV),
         "wg": _rand(gen, (G, hid, d), BF, d ** -0.5), "wu": _rand(gen, (G, hid, d), BF, d ** -0.5),
         "wd": _rand(gen, (G, d, hid), BF, hid ** -0.5)}
    gu = torch.empty((R, 2 * hid), dtype=BF, device=DEV)
    dgu = torch.empty_like(gu)
    t["gate"], t["up"], t["dgate"], t["dup"] = gu[:, :hid], gu[:, hid:], dgu[:, :hid], dgu[:, hid:]
    t["h"], t["dh"] = torch.empty((R, hid), dtype=BF, device=DEV), torch.empty((R, hid), dtype=BF, device=DEV)
    t["y"], t["dx"] = torch.empty((R, d), device=DEV), torch.empty((R, d), device=DEV)
    t["dcoef"] = torch.empty(R, device=DEV)
    for n in ("wg", "wu", "wd"):
        t["d" + n] = torch.empty(t[n].shape, device=DEV)
    return t


def _ffn_step(t, stream=None):
    o, kw = t["off"], {"stream": stream}
    moe.moe_grouped_mm(t["x"], t["wg"], o, t["gate"], **kw)
    moe.moe_grouped_mm(t["x"], t["wu"], o, t["up"], **kw)
    moe.moe_swiglu(t["gate"], t["up"], t["h"], coef=t["coef"], **kw)
    moe.moe_grouped_mm(t["h"], t["wd"], o, t["y"], **kw)
    moe.moe_grouped_wgrad(t["dy"], t["h"], o, t["dwd"], **kw)
    moe.moe_grouped_mm(t["dy"], t["wd"], o, t["dh"], transpose_w=True, **kw)
    moe.moe_swiglu_backward(t["dh"], t["gate"], t["up"], t["dgate"], t["dup"], coef=t["coef"], dcoef=t["dcoef"], **kw)
    moe.moe_grouped_wgrad(t["dgate"], t["x"], o, t["dwg"], **kw)
    moe.moe_grouped_wgrad(t["dup"], t["x"], o, t["dwu"], **kw)
    moe.moe_grouped_mm(t["dgate"], t["wg"], o, t["dx"], transpose_w=True, **kw)
    moe.moe_grouped_mm(t["dup"], t["wu"], o, t["dx"], transpose_w=True, accumulate=True, **kw)


_FFN_OUT = ("y", "dx", "dcoef", "dwg", "dwu", "dwd")


def test_expert_ffn_forward_and_backward():
    """The experts' FFN as a training step runs it, against autograd in 64 bits on the unrounded chain.  Each of the
    two or three bf16 intermediates on a path is off by 2^-8 of its value; as independent relative errors of
    2^-8 / sqrt(3) each, their effect on a sum stays below 3 x 2^-8 of its root mean square."""
    sizes = [0, 40, 1, 130, 300, 0, 7]
    t = _ffn(sizes, 256, 136)
    _ffn_step(t)
    torch.cuda.synchronize()
    assert moe.device_error() == 0
    leaf = {n: t[n].double().requires_grad_() for n in ("x", "coef", "wg", "wu", "wd")}
    off = t["off"].tolist()
    ys = []
    for g in range(len(sizes)):
        s = slice(off[g], off[g + 1])
        a, b = leaf["x"][s] @ leaf["wg"][g].t(), leaf["x"][s] @ leaf["wu"][g].t()
        ys.append((leaf["coef"][s, None] * torch.nn.functional.silu(a) * b) @ leaf["wd"][g].t())
    y = torch.cat(ys)
    y.backward(t["dy"].double())
    ref = {"y": y.detach(), "dx": leaf["x"].grad, "dcoef": leaf["coef"].grad, "dwg": leaf["wg"].grad,
           "dwu": leaf["wu"].grad, "dwd": leaf["wd"].grad}
    for n in _FFN_OUT:
        err = (t[n].double() - ref[n]).square().mean().sqrt()
        assert float(err) <= 3 * 2.0 ** -8 * float(ref[n].square().mean().sqrt()), n


def test_ffn_captured_replayed_and_on_other_streams():
    sizes = [5, 0, 260, 33, 1]
    t, other = _ffn(sizes, 128, 64, seed=1), _ffn(sizes, 128, 64, seed=2)
    _ffn_step(t)
    _ffn_step(other)
    torch.cuda.synchronize()
    want = [t[n].clone() for n in _FFN_OUT], [other[n].clone() for n in _FFN_OUT]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    graphs = []
    for v, s in ((t, s1), (other, s2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            _ffn_step(v, stream=s)
        graphs.append(g)
    for v in (t, other):
        for n in _FFN_OUT:
            v[n].fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):                    # both graphs at once: no buffer is shared
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for v, w in zip((t, other), want):
        for n, r in zip(_FFN_OUT, w):
            assert torch.equal(v[n], r), n   # bit for bit: no atomics, fixed orders
    # new routing in the captured buffers is picked up: everything in the last group
    t["off"].copy_(_offsets([0, 0, 0, 0, sum(sizes)]))
    with torch.cuda.stream(s1):
        graphs[0].replay()
    torch.cuda.synchronize()
    fresh = _ffn(sizes, 128, 64, seed=1)
    fresh["off"] = t["off"]
    _ffn_step(fresh)
    for n in _FFN_OUT:
        assert torch.equal(t[n], fresh[n]), n
    assert moe.device_error() == 0


def test_int8_ffn_against_the_bf16_one():
    """The experts in 8 bits: weights per output channel, activations per row, both products.  A code is off by half
    a step of amax / 127; for normal values amax is about 4 standard deviations at these lengths, so one operand's
    relative error is 4 / 127 / sqrt(12) < 1 %; four operands and SwiGLU stay below 5 % of the output's size."""
    sizes = [3, 90, 0, 20]
    t = _ffn(sizes, 256, 128, seed=4)
    R, d, hid, G = sum(sizes), 256, 128, len(sizes)

    def codes(w):
        q, s = torch.empty(w.shape, dtype=torch.int8, device=DEV), torch.empty(w.shape[:-1], device=DEV)
        moe.moe_quantize_int8(w.reshape(-1, w.shape[-1]), q.view(-1, w.shape[-1]), s.view(-1))
        return q, s

    xq, xs = codes(t["x"])
    for w, y in (("wg", "gate"), ("wu", "up")):
        wq, ws = codes(t[w])
        moe.moe_grouped_mm_int8(xq, xs, wq, ws, t["off"], t[y])
    moe.moe_swiglu(t["gate"], t["up"], t["h"], coef=t["coef"])
    hq, hs = codes(t["h"])
    wq, ws = codes(t["wd"])
    moe.moe_grouped_mm_int8(hq, hs, wq, ws, t["off"], t["y"])
    got = t["y"].double()
    _ffn_step(t)
    err = (got - t["y"].double()).square().mean().sqrt()
    assert float(err) <= 0.05 * float(t["y"].double().square().mean().sqrt())
    assert moe.device_error() == 0


def test_layer_from_the_operators_matches_the_layer():
    """moe_permute's offsets and rows through the grouped products give the routed part of moe_forward.  Where the two
    round to bf16 differs: gate and up here, and h in both (once with its coefficient, once without): four roundings
    of relative error at most u = 2^-8, u / sqrt(3) as a root mean square, independent from element to element.  Each
    enters y linearly (gate's through SiLU, whose relative slope is about 1), so the root mean square of the
    difference is about 2 u / sqrt(3) of y's; 2 u leaves room for the slopes above 1.  The largest of the 150,000
    elements lies some five times further out, so it is not what is tested."""
    from moe_testlib import cfg_of
    from workloads import WORKLOADS, make_inputs
    import dataclasses
    wl = dataclasses.replace(WORKLOADS["tiny"], T=300, x_f32=False, d=512, hidden=256)
    W = {k: v.to(DEV) for k, v in make_inputs(wl, "cpu").items()}
    cfg = cfg_of(wl)
    cfg.n_shared, cfg.shared_hidden = 0, 0
    T, k, E, R = wl.T, wl.top_k, wl.n_experts, wl.T * wl.top_k
    x = W["x"]
    ws = torch.empty(moe.workspace_size(cfg, T), dtype=torch.uint8, device=DEV)
    y = torch.empty((T, wl.d), device=DEV)
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)
    out = {"topk_idx": i32(T, k), "topk_w": torch.empty((T, k), device=DEV), "offsets": i32(E + 1), "src": i32(R)}
    moe.moe_forward(cfg, {n: W[n] for n in ("w_router", "w_gate", "w_up", "w_down")}, x, W["bias"], y, workspace=ws,
                    routing_out=out)
    src = out["src"].long()
    rows = x[src // k].contiguous()
    coef = (out["topk_w"].view(-1)[src] * wl.routed_scale).contiguous()
    gu = torch.empty((R, 2 * wl.hidden), dtype=BF, device=DEV)
    gate, up = gu[:, :wl.hidden], gu[:, wl.hidden:]
    o = torch.empty((R, wl.d), device=DEV)
    off = out["offsets"]
    moe.moe_grouped_mm(rows, W["w_gate"], off, gate)
    moe.moe_grouped_mm(rows, W["w_up"], off, up)
    moe.moe_swiglu(gate, up, gate, coef=coef, n_rows=off[-1:])
    moe.moe_grouped_mm(gate, W["w_down"], off, o)
    got = torch.zeros_like(y).index_add_(0, src // k, o)
    assert moe.device_error() == 0
    assert float((got - y).square().mean().sqrt()) <= 2 * 2.0 ** -8 * float(y.square().mean().sqrt())


def test_outputs_past_two_to_the_31_elements():
    gen = _gen(41)
    rows, n, k = 280_000, 8192, 64                      # y: 2.3e9 elements
    x, w = _rand(gen, (rows, k), BF), _rand(gen, (3, n, k), BF)
    sizes = [100_000, 0, 180_000]
    y = torch.zeros((rows, n), dtype=BF, device=DEV)
    moe.moe_grouped_mm(x, w, _offsets(sizes), y)
    for r in (0, 99_999, 100_000, 262_143, 262_144, rows - 1):
        g = 0 if r < 100_000 else 2
        ref, mag = x[r].double() @ w[g].double().t(), x[r].double().abs() @ w[g].double().abs().t()
        _within(y[r], ref, 66 * 2.0 ** -23 * mag * 1.01 + _eps(BF) * ref.abs(), f"row {r}")
    del y
    dy = _rand(gen, (rows, 2048), BF)
    sizes = [rows // 1000] * 1000 + [0] * 23 + [rows - rows // 1000 * 1000]
    dw = torch.zeros((1024, 2048, 1088), dtype=BF, device=DEV)   # 2.3e9 elements
    x = _rand(gen, (rows, 1088), BF)
    moe.moe_grouped_wgrad(dy, x, _offsets(sizes), dw)
    starts = np.concatenate([[0], np.cumsum(sizes)])
    for g in (0, 500, 963, 964, 999, 1000, 1023):
        a, b = dy[starts[g]:starts[g + 1]].double(), x[starts[g]:starts[g + 1]].double()
        ref, mag = a.t() @ b, a.abs().t() @ b.abs()
        _within(dw[g], ref, 290 * 2.0 ** -23 * mag * 1.01 + _eps(BF) * ref.abs(), f"group {g}")
    assert moe.device_error() == 0


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: no call needs an eager one before it."""
    import os
    import subprocess
    import sys
    code = """
import torch, fine_grained_moe_gemm_b200 as moe
t = lambda *s, d=torch.bfloat16: torch.ones(s, dtype=d, device="cuda")
x, w, wide = t(20, 64), t(2, 48, 64), t(2, 4096, 64)
off = torch.tensor([0, 7, 20], dtype=torch.int32, device="cuda")
big, xb = torch.tensor([0, 3000, 6000], dtype=torch.int32, device="cuda"), t(6000, 64)
y, yb, dw, dwb = t(20, 48), t(6000, 4096), t(2, 48, 64, d=torch.float32), t(2, 4096, 64, d=torch.float32)
q, sx = torch.zeros((20, 64), dtype=torch.int8, device="cuda"), t(20, d=torch.float32)
wq, sw = torch.ones((2, 48, 64), dtype=torch.int8, device="cuda"), t(2, 48, d=torch.float32)
h, dh = t(20, 48), t(20, 48)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    moe.moe_grouped_mm(x, w, off, y)
    moe.moe_grouped_mm(xb, wide, big, yb)
    moe.moe_grouped_wgrad(y, x, off, dw)
    moe.moe_grouped_wgrad(yb, xb, big, dwb)
    moe.moe_swiglu(y, y, h)
    moe.moe_swiglu_backward(dh, y, y, h, dh)
    moe.moe_quantize_int8(x, q, sx)
    moe.moe_grouped_mm_int8(q, sx, wq, sw, off, y)
g.replay()
torch.cuda.synchronize()
assert moe.device_error() == 0
assert float(yb.float().min()) == float(yb.float().max()) == 64.0
assert abs(float(y.float().max()) - 64.0) < 0.5 and float(dw[1].max()) == 13 * 64.0 and float(dwb.max()) == 3000 * 64.0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_many_calls_on_several_streams_at_once():
    """Products of both tilings, gradients and codes interleaved on four streams give the results of calls alone."""
    jobs = []
    for i in range(4):
        gen = _gen(60 + i)
        sizes = [[5, 0, 900, 40], [1, 2, 3], [300] * 6, [0, 2000]][i]
        n, k = [(1032, 520), (72, 2056), (2048, 256), (264, 1024)][i]
        R = sum(sizes)
        j = {"x": _rand(gen, (R, k), BF), "w": _rand(gen, (len(sizes), n, k), BF, 0.1), "dy": _rand(gen, (R, n), BF),
             "off": _offsets(sizes), "y": torch.empty((R, n), device=DEV), "dx": torch.empty((R, k), dtype=BF, device=DEV),
             "dw": torch.empty((len(sizes), n, k), device=DEV), "stream": torch.cuda.Stream()}
        jobs.append(j)

    def call(j, s):
        moe.moe_grouped_mm(j["x"], j["w"], j["off"], j["y"], stream=s)
        moe.moe_grouped_mm(j["dy"], j["w"], j["off"], j["dx"], transpose_w=True, stream=s)
        moe.moe_grouped_wgrad(j["dy"], j["x"], j["off"], j["dw"], stream=s)

    want = []
    for j in jobs:
        call(j, None)
        torch.cuda.synchronize()
        want.append([j[n].clone() for n in ("y", "dx", "dw")])
        for n in ("y", "dx", "dw"):
            j[n].fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for j in jobs:
            call(j, j["stream"])
    torch.cuda.synchronize()
    for j, w in zip(jobs, want):
        for n, r in zip(("y", "dx", "dw"), w):
            assert torch.equal(j[n], r), n
    assert moe.device_error() == 0


def test_ten_thousand_launches_of_narrow_tiles():
    """Tiles of one 64-column block and sums of several rounds of the ring, back to back: no wait may run out and no
    launch may differ.  (A loading warp without bytes in such tiles once fell two rounds behind and waited for a phase
    that was over, about once in a million launches.)"""
    gen = _gen(77)
    cases = []
    for sizes, n, k in (([535], 192, 5648), ([700, 3, 1500], 136, 264), ([9000], 72, 64)):
        dy, x = _rand(gen, (sum(sizes), n), FH), _rand(gen, (sum(sizes), k), FH)
        cases.append((dy, x, _offsets(sizes), torch.empty((len(sizes), n, k), device=DEV)))
    for dy, x, off, dw in cases:
        moe.moe_grouped_wgrad(dy, x, off, dw)
        want = dw.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(250):
                moe.moe_grouped_wgrad(dy, x, off, dw)
        for _ in range(14):
            g.replay()
            assert moe.device_error() == 0
        assert torch.equal(dw, want)


def test_binding_refusals_on_the_gpu():
    x, w = torch.zeros((4, 16), dtype=BF, device=DEV), torch.zeros((2, 8, 16), dtype=BF, device=DEV)
    off, y = torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros((4, 8), dtype=BF, device=DEV)
    ok = lambda **kw: moe.moe_grouped_mm(**{**dict(x=x, w=w, offsets=off, y=y), **kw})
    ok()
    for bad in (dict(x=x[:, :8]), dict(x=x.half()), dict(x=x.t()), dict(w=w[0]), dict(w=w.float()), dict(offsets=off.long()),
                dict(offsets=off[:2]), dict(offsets=None), dict(y=y.half()), dict(y=y[:3]), dict(x=x.cpu()),
                dict(w=w.transpose(1, 2)), dict(y=y[:, :1].expand(4, 8))):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(moe.MoeError):      # rows that are not 16 bytes apart
        ok(x=torch.zeros((4, 20), dtype=BF, device=DEV)[:, :16])
    with pytest.raises(moe.MoeError):      # rows that lie on one another
        ok(x=torch.zeros((1, 16), dtype=BF, device=DEV).expand(4, 16))
    with pytest.raises(moe.MoeError):      # a sum of 12
        ok(x=torch.zeros((4, 12), dtype=BF, device=DEV), w=torch.zeros((2, 8, 12), dtype=BF, device=DEV))
    assert moe.device_error() == 0
