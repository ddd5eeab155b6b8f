"""The experts' products and what stands around them in training and in 8-bit serving: what is measured.

Five operators work on rows sorted by expert ("groups"; ``offsets[g] .. offsets[g + 1]`` are group g's rows):

  grouped product       y[r, n] = sum_k x[r, k] w[g(r), n, k]         (the projections)
                        y[r, n] = sum_k x[r, k] w[g(r), k, n]         (their input gradients)
  weight gradient       dw[g, n, k] = sum_{r in g} dy[r, n] x[r, k]
  SwiGLU                h = c silu(a) b for each row's coefficient c, and the gradients of a, b and c
  int8 codes            sx[r] = max_k |x[r, k]| / 127 (1 for a row of zeros), q = nearest integer of x / sx,
                        ties to even
  int8 grouped product  y[r, n] = sx[r] sw[g(r), n] sum_k q[r, k] w[g(r), n, k]

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits (64 where 32 lose exact
integers or decide a rounding), else it calls the framework.  The widths, expert counts and batches are those of
this repository's workloads (tiny, decode, prefill, skewed, its dense FFN of width 18432), or generic.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def _moe():
    import fine_grained_moe_gemm_b200 as moe
    return moe


def listed():
    return [
        # the tiny workload: 64 tokens x 4 of 16 experts, first projection; a call's latency
        {"name": "mm_tiny", "op": "mm", "groups": 16, "rows": 256, "spare": 0, "n": 128, "k": 256, "zipf": 0.0,
         "transpose": False, "type": "bf16", "out": "f32"},
        # decode, 128 tokens x 8 of 256 experts: four rows an expert, every expert's weights are read
        {"name": "mm_decode", "op": "mm", "groups": 256, "rows": 1024, "spare": 0, "n": 2048, "k": 7168, "zipf": 0.0,
         "transpose": False, "type": "bf16", "out": "bf16"},
        # the input gradient of the first projection over a 4096-token batch, uneven experts, padded buffer
        {"name": "mm_prefill_dx", "op": "mm", "groups": 256, "rows": 32768, "spare": 1000, "n": 7168, "k": 2048,
         "zipf": 0.5, "transpose": True, "type": "bf16", "out": "bf16"},
        # the down projection of a 16384-token batch with hot experts: 131072 rows, bound by the tensor cores
        {"name": "mm_skewed", "op": "mm", "groups": 256, "rows": 131072, "spare": 0, "n": 7168, "k": 2048,
         "zipf": 1.2, "transpose": False, "type": "bf16", "out": "bf16"},
        # ragged experts of odd widths in half precision, gradients kept in 32 bits
        {"name": "wgrad_odd", "op": "wgrad", "groups": 24, "rows": 5003, "spare": 13, "n": 1032, "k": 1160,
         "zipf": 0.8, "type": "f16", "out": "f32"},
        # the first projection's weight gradient over a 4096-token batch: 256 gradients of 29 MB
        {"name": "wgrad_prefill", "op": "wgrad", "groups": 256, "rows": 32768, "spare": 0, "n": 2048, "k": 7168,
         "zipf": 0.5, "type": "bf16", "out": "bf16"},
        # decode: the gate and up halves of one buffer
        {"name": "swiglu_decode", "op": "swiglu", "rows": 1024, "h": 2048, "coef": True, "type": "bf16"},
        # the backward pass over a 16384-token batch with the routing weights' gradient
        {"name": "swiglu_backward", "op": "swiglu_backward", "rows": 131072, "h": 2048, "coef": True, "type": "bf16"},
        # codes of a decode batch, and of a prompt of 16384 tokens
        {"name": "int8_decode", "op": "quantize", "rows": 128, "k": 7168, "type": "bf16"},
        {"name": "int8_prompt", "op": "quantize", "rows": 16384, "k": 7168, "type": "bf16"},
        # the dense FFN's down projection for sixteen tokens: one group, a long sum, few rows
        {"name": "mm_int8_dense", "op": "mm_int8", "groups": 1, "rows": 16, "spare": 0, "n": 7168, "k": 18432,
         "zipf": 0.0, "out": "bf16"},
        # the first projection over an 8192-token batch with 8-bit experts
        {"name": "mm_int8_prefill", "op": "mm_int8", "groups": 256, "rows": 65536, "spare": 0, "n": 2048, "k": 7168,
         "zipf": 0.5, "out": "bf16"},
    ]


_MOST_WEIGHTS = 256 * 2048 * 7168   # elements of all groups' weights
_MOST_MACS = 131072 * 2048 * 7168


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mm", "mm", "wgrad", "swiglu", "swiglu_backward", "quantize", "mm_int8", "mm_int8"])
    if op in ("swiglu", "swiglu_backward"):
        return {"op": op, "rows": _log(rng, 1, 131072), "h": 8 * _log(rng, 8, 256), "coef": rng.random() < 0.7,
                "type": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 16384), "k": 16 * _log(rng, 4, 448),
                "type": rng.choice(["bf16", "bf16", "f16", "f32"])}
    step = 16 if op == "mm_int8" else 8   # of the summed width: rows of 16 bytes
    while True:
        groups = rng.choice([1, _log(rng, 2, 256)])
        rows, n, k = _log(rng, 1, 131072), 8 * _log(rng, 8, 896), step * _log(rng, 64 // step, 7168 // step)
        if groups == 1 and rng.random() < 0.3:
            k = 18432
        # fp32 results of a gradient are twice as many bytes as the largest listed case's
        if groups * n * k <= _MOST_WEIGHTS // 2 and rows * n * k <= _MOST_MACS:
            break
    case = {"op": op, "groups": groups, "rows": rows, "spare": rng.choice([0, rng.randrange(1, 200)]), "n": n, "k": k,
            "zipf": rng.choice([0.0, 0.5, 1.2])}
    if op == "mm":
        case["transpose"] = rng.random() < 0.5
    if op != "mm_int8":
        case["type"] = rng.choice(["bf16", "bf16", "f16"])
    case["out"] = rng.choice([case.get("type", "bf16"), "f32"])
    return case


def _sizes(case):
    """Rows of each group, the same for every seed but for their order: the case's rows thrown over its groups."""
    g = case["groups"]
    p = np.arange(1, g + 1, dtype=np.float64) ** -case["zipf"]
    return np.random.default_rng([g, case["rows"], int(case["zipf"] * 10)]).multinomial(case["rows"], p / p.sum())


def _normal(gen, shape, std, dtype):
    """Normal values in slices, so that the largest tensors need little room besides their own."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(shape[0], -1)
    step = max(1, (1 << 28) // flat.shape[1])
    for i in range(0, shape[0], step):
        part = torch.randn(flat[i:i + step].shape, generator=gen, device="cuda")
        flat[i:i + step] = part.mul_(std)
    return out


def _codes(gen, shape):
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = out.view(shape[0], -1)
    step = max(1, (1 << 28) // flat.shape[1])
    for i in range(0, shape[0], step):
        part = torch.randn(flat[i:i + step].shape, generator=gen, device="cuda")
        flat[i:i + step] = part.mul_(36.0).round_().clamp_(-127, 127)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op, rows = case["op"], case["rows"]
    if op in ("swiglu", "swiglu_backward"):
        t, h = _TYPES[case["type"]], case["h"]
        both = _normal(gen, (rows, 2 * h), 1.5, t)
        s["gate"], s["up"] = both[:, :h], both[:, h:]
        s["coef"] = torch.rand(rows, generator=gen, device="cuda") if case["coef"] else None
        if op == "swiglu":
            s["h"] = torch.empty((rows, h), dtype=t, device="cuda")
        else:
            s["dh"] = _normal(gen, (rows, h), 0.1, t)
            grads = torch.empty((rows, 2 * h), dtype=t, device="cuda")
            s["dgate"], s["dup"] = grads[:, :h], grads[:, h:]
            s["dcoef"] = torch.empty(rows, device="cuda") if case["coef"] else None
        return s
    if op == "quantize":
        k = case["k"]
        x = _normal(gen, (rows, k), 1.0, torch.float32)
        x[:, torch.randint(k, (4,), generator=gen, device="cuda")] *= 20.0   # the few wide channels of real activations
        s["x"] = x.to(_TYPES[case["type"]])
        s["q"] = torch.empty((rows, k), dtype=torch.int8, device="cuda")
        s["sx"] = torch.empty(rows, device="cuda")
        return s
    g, n, k = case["groups"], case["n"], case["k"]
    sizes = np.random.default_rng(seed).permutation(_sizes(case))
    ends = np.concatenate([[0], np.cumsum(sizes)])
    s["ends"] = ends.tolist()
    s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    room = rows + case["spare"]
    if op == "mm":
        t = _TYPES[case["type"]]
        s["x"] = _normal(gen, (room, k), 1.0, t)
        s["w"] = _normal(gen, (g, k, n) if case["transpose"] else (g, n, k), 0.02, t)
        s["y"] = torch.zeros((room, n), dtype=_TYPES[case["out"]], device="cuda")
    elif op == "wgrad":
        t = _TYPES[case["type"]]
        s["dy"] = _normal(gen, (room, n), 0.1, t)
        s["x"] = _normal(gen, (room, k), 1.0, t)
        s["dw"] = torch.empty((g, n, k), dtype=_TYPES[case["out"]], device="cuda")
    else:
        s["q"] = _codes(gen, (room, k))
        s["sx"] = torch.rand(room, generator=gen, device="cuda").mul_(0.05).add_(0.01)
        s["w"] = _codes(gen, (g, n, k))
        s["sw"] = torch.rand((g, n), generator=gen, device="cuda").mul_(1e-3).add_(1e-4)
        s["y"] = torch.zeros((room, n), dtype=_TYPES[case["out"]], device="cuda")
    return s


def _padded(case, ends):
    """Each group's rows as one padded block (row numbers, and which of them are rows of the group), where padding
    costs little: many small groups of like size.  None where it would cost more than a product for each group."""
    sizes = np.diff(ends)
    most = max(int(sizes.max()), 1)
    if case["groups"] == 1 or most * case["groups"] > 4 * case["rows"] + 64 * case["groups"]:
        return None
    at = torch.arange(most, device="cuda")
    starts, counts = torch.tensor(ends[:-1], device="cuda"), torch.tensor(sizes, device="cuda")
    real = at < counts[:, None]
    return (starts[:, None] + at).where(real, torch.zeros_like(at)), real


def _run_own(s):
    moe, case = _moe(), s["case"]
    op = case["op"]
    if op == "mm":
        moe.moe_grouped_mm(s["x"], s["w"], s["offsets"], s["y"], transpose_w=case["transpose"])
        return s["y"]
    if op == "wgrad":
        moe.moe_grouped_wgrad(s["dy"], s["x"], s["offsets"], s["dw"])
        return s["dw"]
    if op == "swiglu":
        moe.moe_swiglu(s["gate"], s["up"], s["h"], coef=s["coef"])
        return s["h"]
    if op == "swiglu_backward":
        moe.moe_swiglu_backward(s["dh"], s["gate"], s["up"], s["dgate"], s["dup"], coef=s["coef"], dcoef=s["dcoef"])
        return [s["dgate"], s["dup"]] + ([s["dcoef"]] if case["coef"] else [])
    if op == "quantize":
        moe.moe_quantize_int8(s["x"], s["q"], s["sx"])
        return [s["q"], s["sx"]]
    moe.moe_grouped_mm_int8(s["q"], s["sx"], s["w"], s["sw"], s["offsets"], s["y"])
    return s["y"]


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op = case["op"]
    if op == "swiglu":
        a, b = s["gate"].float(), s["up"].float()
        y = a * torch.sigmoid(a) * b
        return (y * s["coef"][:, None] if case["coef"] else y).to(s["h"].dtype)
    if op == "swiglu_backward":
        a, b, dh = s["gate"].float(), s["up"].float(), s["dh"].float()
        sig = torch.sigmoid(a)
        act = a * sig
        dy = dh * s["coef"][:, None] if case["coef"] else dh
        out = [(dy * b * (sig + act * (1.0 - sig))).to(s["dgate"].dtype), (dy * act).to(s["dup"].dtype)]
        return out + ([(dh * act * b).sum(1)] if case["coef"] else [])
    if op == "quantize":
        # the quotient in 64 bits: in 32 it can round onto the border between two codes
        x = s["x"].float()
        sx = x.abs().amax(1) / 127.0
        sx = torch.where(sx == 0.0, torch.ones_like(sx), sx)
        return [torch.round(x.double() / sx.double()[:, None]).to(torch.int8), sx]
    ends = s["ends"]
    block = _padded(case, ends)
    if op == "wgrad":
        dy, x, dw = s["dy"], s["x"], s["dw"]
        if block is not None:
            idx, real = block
            dyb = dy[idx].float() * real[:, :, None]
            dw[...] = torch.bmm(dyb.transpose(1, 2), x[idx].float())
            return dw
        for g in range(case["groups"]):   # ragged: one product for each group
            a, b = ends[g], ends[g + 1]
            dw[g] = dy[a:b].float().t() @ x[a:b].float()
        return dw
    y = s["y"]
    if op == "mm":
        x, w = s["x"], s["w"] if case["transpose"] else s["w"].transpose(1, 2)
        if block is not None:
            idx, real = block
            y[idx[real]] = torch.bmm(x[idx].float(), w.float())[real].to(y.dtype)
            return y
        for g in range(case["groups"]):
            a, b = ends[g], ends[g + 1]
            if b > a:
                y[a:b] = x[a:b].float() @ w[g].float()
        return y
    q, sx, w, sw = s["q"], s["sx"], s["w"], s["sw"]
    for g in range(case["groups"]):       # sums of integers past 2^24: in 64 bits
        a, b = ends[g], ends[g + 1]
        if b > a:
            acc = q[a:b].double() @ w[g].double().t()
            y[a:b] = acc.float() * sx[a:b, None] * sw[g]
    return y


def work(case):
    op, rows = case["op"], case["rows"]
    if op in ("swiglu", "swiglu_backward"):
        e, h = _BYTES[case["type"]], case["h"]
        c = 4 * rows if case["coef"] else 0
        if op == "swiglu":
            return {"bytes": 3 * rows * h * e + c, "flops": 6 * rows * h}
        return {"bytes": 5 * rows * h * e + 2 * c, "flops": 14 * rows * h}
    if op == "quantize":
        return {"bytes": rows * case["k"] * (_BYTES[case["type"]] + 1) + 4 * rows, "flops": 4 * rows * case["k"]}
    g, n, k = case["groups"], case["n"], case["k"]
    used = int((_sizes(case) > 0).sum())
    out = _BYTES[case["out"]]
    flops = 2 * rows * n * k
    if op == "mm":
        e = _BYTES[case["type"]]
        return {"bytes": used * n * k * e + rows * k * e + rows * n * out, "flops": flops}
    if op == "wgrad":
        return {"bytes": rows * (n + k) * _BYTES[case["type"]] + g * n * k * out, "flops": flops}
    return {"bytes": used * n * (k + 4) + rows * (k + 4) + rows * n * out, "flops": flops}


def exact(case, seed):
    """The definitions in 64 bits, group by group (elementwise ones in slices of rows)."""
    s = prepare(case, seed)
    op, rows = case["op"], case["rows"]
    if op in ("swiglu", "swiglu_backward"):
        h = case["h"]
        f64 = dict(dtype=torch.float64, device="cuda")
        first, second, third = torch.empty((rows, h), **f64), torch.empty((rows, h), **f64), torch.empty(rows, **f64)
        step = max(1, (1 << 26) // h)
        for i in range(0, rows, step):
            j = slice(i, i + step)
            a, b = s["gate"][j].double(), s["up"][j].double()
            c = s["coef"][j].double()[:, None] if case["coef"] else torch.ones_like(a[:, :1])
            sig = 1.0 / (1.0 + torch.exp(-a))
            if op == "swiglu":
                first[j] = c * (a * sig) * b
                continue
            dh = s["dh"][j].double()
            first[j] = dh * c * b * (sig * (1.0 + a * (1.0 - sig)))
            second[j] = dh * c * (a * sig)
            third[j] = torch.einsum("rh,rh,rh->r", dh, a * sig, b)
        if op == "swiglu":
            return first
        return [first, second] + ([third] if case["coef"] else [])
    if op == "quantize":
        # the scale is a number of 32 bits by definition, and the codes go by that number
        sx = (s["x"].double().abs().max(dim=1).values / 127.0).float()
        sx[sx == 0.0] = 1.0
        return [torch.round(s["x"].double() / sx.double().unsqueeze(1)).to(torch.int8), sx.double()]
    ends, n, k = s["ends"], case["n"], case["k"]
    if op == "wgrad":
        dw = torch.zeros((case["groups"], n, k), dtype=torch.float64, device="cuda")
        for g, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
            torch.mm(s["dy"][a:b].double().t(), s["x"][a:b].double(), out=dw[g])
        return dw
    y = torch.zeros((rows + case["spare"], n), dtype=torch.float64, device="cuda")
    for g, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        if b == a:
            continue
        if op == "mm":
            w = s["w"][g].double()
            y[a:b] = torch.mm(s["x"][a:b].double(), w if case["transpose"] else w.t())
        else:
            scaled = s["w"][g].double() * s["sw"][g].double()[:, None]
            y[a:b] = torch.mm(s["q"][a:b].double() * s["sx"][a:b].double()[:, None], scaled.t())
    return y
