"""The experts' own work between the gather and the combine, as cases to measure.

Three operators that run over rows sorted by expert:

* ``product``: every row times its expert's matrix, in 16 bits, for segments of
  any length; with ``grad`` also the gradients of the rows and of the matrices;
* ``product8``: the same of e4m3 values with a scale per 128 of a row and per
  128 x 128 of a matrix, for segments or for one matrix; with ``grad`` also the
  product that takes a gradient in e4m3 back to the rows;
* ``act`` / ``act_grad``: silu of a row's first half times its second half, in
  16 bits or in e4m3 with scales (or e4m3 alone, of rows as they are), and the
  gradient.

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with the calls of ``message_fp16_all_amd.hr``.
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
_F8 = torch.float8_e4m3fn
_F8_MAX = 448.0
_F32_MIN = 2.0 ** -126
_GROUP = 128


def listed():
    return [
        # one decoded token, two of whose picks are among this rank's sixteen experts: latency, and two matrices
        dict(name="product 2x4096x2048", op="product", dtype="f16", rows=2, k=4096, n=2048, experts=16, pad=1,
             transposed=False, grad=False),
        # a decode batch, 64 tokens of 8 picks: every matrix is read for about 8 rows
        dict(name="product 512x5120x2560", op="product", dtype="bf16", rows=512, k=5120, n=2560, experts=64, pad=16,
             transposed=False, grad=False),
        # an odd prefill batch of 8191 tokens and 8 picks over 128 experts
        dict(name="product 65528x4096x2048", op="product", dtype="bf16", rows=65528, k=4096, n=2048, experts=128,
             pad=1, transposed=False, grad=False),
        # a training step, there and back: 4096 tokens of 4 picks, segments padded to a product's tile
        dict(name="product 16384x4096x4096 grad", op="product", dtype="f16", rows=16384, k=4096, n=4096, experts=32,
             pad=128, transposed=False, grad=True),
        # odd widths, matrices kept the other way round
        dict(name="product 2151x1327x1001 grad", op="product", dtype="bf16", rows=2151, k=1327, n=1001, experts=8,
             pad=1, transposed=True, grad=True),
        # one decoded token through a dense layer in 8 bits
        dict(name="product8 1x8192x10240", op="product8", dtype="bf16", rows=1, k=8192, n=10240, experts=1, pad=1,
             grad=False),
        # a decode batch over experts in 8 bits
        dict(name="product8 384x5120x5120", op="product8", dtype="f16", rows=384, k=5120, n=5120, experts=64, pad=16,
             grad=False),
        # a prefill chunk through a dense layer in 8 bits
        dict(name="product8 8192x8192x8192", op="product8", dtype="bf16", rows=8192, k=8192, n=8192, experts=1, pad=1,
             grad=False),
        # a ragged training batch in 8 bits: there, and the rows' gradient
        dict(name="product8 32764x4096x4096 grad", op="product8", dtype="bf16", rows=32764, k=4096, n=4096,
             experts=64, pad=1, grad=True),
        # one decoded token's eight rows: latency alone
        dict(name="act 8x2048", op="act", dtype="f16", rows=8, width=2048, gated=True, out=True, codes=False),
        # a prefill batch's rows straight into an 8-bit product
        dict(name="act 65528x2048 e4m3", op="act", dtype="bf16", rows=65528, width=2048, gated=True, out=False,
             codes=True),
        # a training step: the gradient, and the activation once more for the weights' gradient
        dict(name="act_grad 16383x4096", op="act_grad", dtype="f16", rows=16383, width=4096, out=True),
    ]


def _spread(rng, low, high):
    """A whole number spread over the logarithm: a power of two or an odd one."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    if rng.random() < 0.4:
        return max(low, 1 << int(math.log2(v)))
    return min(high, int(v) | 1)


def _width(rng, low=64, high=10240):
    """A row length: mostly a multiple of 64 or a power of two, sometimes odd."""
    if rng.random() < 0.2:
        return _spread(rng, low, high)
    return rng.choice([1 << rng.randint(int(math.log2(low)), int(math.log2(high))),
                       64 * _spread(rng, -(-low // 64), high // 64)])


def draw(rng):
    op = rng.choice(["product", "product", "product8", "product8", "act", "act_grad"])
    most = [work(c) for c in listed() if c["op"] == op]
    most = {what: max(w[what] for w in most) for what in ("bytes", "flops")}
    while True:
        if op in ("product", "product8"):
            case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), rows=_spread(rng, 1, 65536), k=_width(rng),
                        n=_width(rng), experts=rng.choice([1, 2, 4, 8, 16, 32, 60, 64, 96, 128, 160, 256]),
                        pad=rng.choice([1, 1, 16, 64, 128]), grad=rng.random() < 0.4)
            if op == "product":
                case["transposed"] = rng.random() < 0.3
            if _capacity(case) > 2 * 65536:
                continue
        elif op == "act":
            out = rng.random() < 0.6
            case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), rows=_spread(rng, 1, 65536), width=_width(rng),
                        gated=rng.random() < 0.75, out=out, codes=not out or rng.random() < 0.3)
            if not case["gated"]:
                case["out"], case["codes"] = False, True
        else:
            case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), rows=_spread(rng, 1, 65536), width=_width(rng),
                        out=rng.random() < 0.5)
        w = work(case)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return case


def _capacity(case):
    """Rows that the sorted rows take at most: every segment that holds one is rounded up."""
    return case["rows"] + min(case["experts"], case["rows"]) * (case["pad"] - 1)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    {"product": _prepare_product, "product8": _prepare_product8, "act": _prepare_act,
     "act_grad": _prepare_act_grad}[case["op"]](case, g, state)
    return state


def _normal(g, *shape, sigma=1.0, dtype=torch.float32):
    x = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)
    return x.mul_(sigma) if sigma != 1.0 else x


def _segments(case, g, s):
    """The rows of every expert, some of them liked more than others; the offsets on the GPU, as a sort leaves
    them, and on the host; and a mask of the rows that are not padding."""
    rows, E, pad = case["rows"], case["experts"], case["pad"]
    e = (_normal(g, rows, E) + 0.5 * _normal(g, E)).argmax(1)
    count = torch.bincount(e, minlength=E).cpu().tolist()
    bounds = [0]
    here = torch.zeros(_capacity(case), 1, dtype=torch.bool, device="cuda")
    for c in count:
        here[bounds[-1]:bounds[-1] + c] = True
        bounds.append(bounds[-1] + -(-c // pad) * pad)
    s["bounds"] = bounds
    s["offsets"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    return here


def _prepare_product(case, g, s):
    k, n, E, dt = case["k"], case["n"], case["experts"], _TYPES[case["dtype"]]
    here = _segments(case, g, s)
    rows = here.shape[0]
    s["x"] = _normal(g, rows, k, dtype=dt) * here                 # padding rows are zeros, as a gather writes them
    s["w"] = _normal(g, *((E, k, n) if case["transposed"] else (E, n, k)), sigma=k ** -0.5, dtype=dt)
    s["out"] = torch.zeros(rows, n, dtype=dt, device="cuda")
    if case["grad"]:
        s["dy"] = _normal(g, rows, n, sigma=0.1, dtype=dt) * here
        s["dx"] = torch.zeros_like(s["x"])
        s["dw"] = torch.empty_like(s["w"])


def _codes(x, rows):
    """(e4m3 codes, scales) of x with a scale per ``rows`` rows and 128 columns."""
    r, c = x.shape
    nr, nc = -(-r // rows), -(-c // _GROUP)
    whole = torch.zeros(nr * rows, nc * _GROUP, device="cuda")
    whole[:r, :c] = x
    whole = whole.view(nr, rows, nc, _GROUP)
    scales = (whole.abs().amax((1, 3)) / _F8_MAX).clamp_min(_F32_MIN)
    codes = (whole / scales[:, None, :, None]).view(nr * rows, -1)[:r, :c].contiguous().to(_F8)
    return codes, scales


def _prepare_product8(case, g, s):
    k, n, E, dt = case["k"], case["n"], case["experts"], _TYPES[case["dtype"]]
    here = _segments(case, g, s)
    rows = here.shape[0]

    def some(width, sigma):
        # a few channels stand out, so that the groups' scales differ
        v = _normal(g, rows, width, sigma=sigma)
        v[:, ::97] *= 8
        codes, scales = _codes(v, 1)
        return (codes.view(torch.uint8) * here).view(_F8), scales * here

    s["x"], s["x_scales"] = some(k, 1.0)
    s["w"] = torch.empty(E, n, k, dtype=_F8, device="cuda")
    s["w_scales"] = torch.empty(E, -(-n // _GROUP), -(-k // _GROUP), device="cuda")
    for e in range(E):
        s["w"][e], s["w_scales"][e] = _codes(_normal(g, n, k, sigma=k ** -0.5), _GROUP)
    s["out"] = torch.zeros(rows, n, dtype=dt, device="cuda")
    if case["grad"]:
        s["dy"], s["dy_scales"] = some(n, 0.1)
        s["dx"] = torch.zeros(rows, k, dtype=dt, device="cuda")


def _prepare_act(case, g, s):
    rows, width, dt = case["rows"], case["width"], _TYPES[case["dtype"]]
    s["x"] = _normal(g, rows, width * (2 if case["gated"] else 1), sigma=1.5, dtype=dt)
    s["out"] = torch.empty(rows, width, dtype=dt, device="cuda") if case["out"] else None
    s["codes"] = torch.empty(rows, width, dtype=_F8, device="cuda") if case["codes"] else None
    s["scales"] = torch.empty(rows, -(-width // _GROUP), device="cuda") if case["codes"] else None


def _prepare_act_grad(case, g, s):
    rows, width, dt = case["rows"], case["width"], _TYPES[case["dtype"]]
    s["x"] = _normal(g, rows, 2 * width, sigma=1.5, dtype=dt)
    s["dy"] = _normal(g, rows, width, sigma=0.1, dtype=dt)
    s["dx"] = torch.empty_like(s["x"])
    s["out"] = torch.empty_like(s["dy"]) if case["out"] else None


# --------------------------------------------------------------------- run

_hr = None


def run(state):
    global _hr
    op = state["case"]["op"]
    if not own:
        return _PLAIN[op](state)
    if _hr is None:
        from message_fp16_all_amd import hr
        _hr = hr
    return _OWN[op](state)


def _own_product(s):
    c = s["case"]
    other = c["transposed"]
    _hr.experts_product(s["x"], s["w"], s["out"], offsets=s["offsets"], transposed=other)
    if not c["grad"]:
        return {"out": s["out"]}
    _hr.experts_product(s["dy"], s["w"], s["dx"], offsets=s["offsets"], transposed=not other)
    a, b = (s["x"], s["dy"]) if other else (s["dy"], s["x"])
    _hr.experts_product_grad(a, b, s["dw"], offsets=s["offsets"])
    return {"out": s["out"], "dx": s["dx"], "dw": s["dw"]}


def _own_product8(s):
    _hr.experts_product(s["x"], s["w"], s["out"], offsets=s["offsets"], x_scales=s["x_scales"],
                        w_scales=s["w_scales"])
    if not s["case"]["grad"]:
        return {"out": s["out"]}
    _hr.experts_product(s["dy"], s["w"], s["dx"], offsets=s["offsets"], x_scales=s["dy_scales"],
                        w_scales=s["w_scales"], transposed=True)
    return {"out": s["out"], "dx": s["dx"]}


def _own_act(s):
    _hr.experts_act(s["x"], s["out"], gated=s["case"]["gated"], out8=s["codes"], scales=s["scales"])
    return {"out": s["out"], "codes": s["codes"], "scales": s["scales"]}


def _own_act_grad(s):
    _hr.experts_act_grad(s["dy"], s["x"], s["dx"], out=s["out"])
    return {"dx": s["dx"], "out": s["out"]}


_OWN = {"product": _own_product, "product8": _own_product8, "act": _own_act, "act_grad": _own_act_grad}


# ------------------------------------------------------------- plain forms

def _each(s):
    """(expert, first row, row after the last) of the segments that hold any."""
    b = s["bounds"]
    return [(e, b[e], b[e + 1]) for e in range(len(b) - 1) if b[e + 1] > b[e]]


def _plain_product(s):
    c = s["case"]
    out = torch.zeros_like(s["out"])
    grads = {}
    if c["grad"]:
        grads = {"dx": torch.zeros_like(s["dx"]), "dw": torch.zeros_like(s["dw"])}
    for e, a, b in _each(s):
        w = s["w"][e].float()
        if not c["transposed"]:
            w = w.t()                                             # k x n
        x = s["x"][a:b].float()
        out[a:b] = (x @ w).to(out.dtype)
        if c["grad"]:
            dy = s["dy"][a:b].float()
            grads["dx"][a:b] = (dy @ w.t()).to(out.dtype)
            grads["dw"][e] = (x.t() @ dy if c["transposed"] else dy.t() @ x).to(out.dtype)
    return {"out": out, **grads}


def _wide(codes, scales):
    """What codes with a scale per 128 columns stand for."""
    return codes.float() * scales.repeat_interleave(_GROUP, 1)[:, :codes.shape[1]]


def _plain_product8(s):
    c = s["case"]
    out = {"out": torch.zeros_like(s["out"])}
    if c["grad"]:
        out["dx"] = torch.zeros_like(s["dx"])
    for e, a, b in _each(s):
        w = _wide(s["w"][e], s["w_scales"][e].repeat_interleave(_GROUP, 0)[:c["n"]])
        out["out"][a:b] = (_wide(s["x"][a:b], s["x_scales"][a:b]) @ w.t()).to(s["out"].dtype)
        if c["grad"]:
            out["dx"][a:b] = (_wide(s["dy"][a:b], s["dy_scales"][a:b]) @ w).to(s["out"].dtype)
    return out


def _plain_act(s):
    c = s["case"]
    x = s["x"].float()
    if c["gated"]:
        gate, up = x[:, :c["width"]], x[:, c["width"]:]
        x = gate / (1.0 + torch.exp(-gate)) * up
    codes, scales = _codes(x, 1) if c["codes"] else (None, None)
    return {"out": x.to(s["x"].dtype) if c["out"] else None, "codes": codes, "scales": scales}


def _plain_act_grad(s):
    c = s["case"]
    x, dy, dt = s["x"].float(), s["dy"].float(), s["x"].dtype
    gate, up = x[:, :c["width"]], x[:, c["width"]:]
    sig = 1.0 / (1.0 + torch.exp(-gate))
    silu = gate * sig
    dx = torch.cat([dy * up * (sig + silu * (1.0 - sig)), dy * silu], 1).to(dt)
    return {"dx": dx, "out": (silu * up).to(dt) if c["out"] else None}


_PLAIN = {"product": _plain_product, "product8": _plain_product8, "act": _plain_act, "act_grad": _plain_act_grad}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The same from the definitions in 64 bits, before the last rounding to a type."""
    s = prepare(case, seed)
    return {"product": _exact_product, "product8": _exact_product8, "act": _exact_act,
            "act_grad": _exact_act_grad}[case["op"]](case, s)


def _exact_product(c, s):
    f64 = dict(dtype=torch.float64, device="cuda")
    rows, E = s["x"].shape[0], c["experts"]
    out = {"out": torch.zeros(rows, c["n"], **f64)}
    if c["grad"]:
        out["dx"] = torch.zeros(rows, c["k"], **f64)
        out["dw"] = torch.zeros(s["w"].shape, **f64)
    ends = s["offsets"].tolist()
    for e in range(E):
        seg = slice(ends[e], ends[e + 1])
        w = s["w"][e].double()
        to_out, to_dw = ("rk,kn->rn", "rk,rn->kn") if c["transposed"] else ("rk,nk->rn", "rk,rn->nk")
        to_dx = "rn,kn->rk" if c["transposed"] else "rn,nk->rk"
        x = s["x"][seg].double()
        out["out"][seg] = torch.einsum(to_out, x, w)
        if c["grad"]:
            dy = s["dy"][seg].double()
            out["dx"][seg] = torch.einsum(to_dx, dy, w)
            out["dw"][e] = torch.einsum(to_dw, x, dy)
    return out


def _exact_product8(c, s):
    # one group of 128 of the contraction after another, its products times its scales
    f64 = dict(dtype=torch.float64, device="cuda")
    rows = s["x"].shape[0]
    out = {"out": torch.zeros(rows, c["n"], **f64)}
    if c["grad"]:
        out["dx"] = torch.zeros(rows, c["k"], **f64)
    ends = s["offsets"].tolist()
    for e in range(c["experts"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        w, ws = s["w"][e].double(), s["w_scales"][e].double()
        for j in range(ws.shape[1]):
            cols = slice(j * _GROUP, min(c["k"], (j + 1) * _GROUP))
            per_row = ws[:, j].repeat_interleave(_GROUP)[:c["n"]]
            p = s["x"][a:b, cols].double() @ w[:, cols].t()
            out["out"][a:b] += p * per_row * s["x_scales"][a:b, j, None].double()
        if c["grad"]:
            for j in range(ws.shape[0]):
                cols = slice(j * _GROUP, min(c["n"], (j + 1) * _GROUP))
                per_col = ws[j].repeat_interleave(_GROUP)[:c["k"]]
                p = s["dy"][a:b, cols].double() @ w[cols]
                out["dx"][a:b] += p * per_col * s["dy_scales"][a:b, j, None].double()
    return out


def _exact_act(c, s):
    y = s["x"].double()
    if c["gated"]:
        gate, up = y.split(c["width"], dim=1)
        y = gate * torch.sigmoid(gate) * up
    codes = scales = None
    if c["codes"]:
        parts = y.split(_GROUP, dim=1)
        scales = torch.stack([p.abs().max(dim=1).values for p in parts], 1) / _F8_MAX
        codes = torch.cat([p / scales[:, i:i + 1] for i, p in enumerate(parts)], 1)
    return {"out": y if c["out"] else None, "codes": codes, "scales": scales}


def _exact_act_grad(c, s):
    # the derivative of sum(dy * silu(gate) * up), silu'(g) = sigmoid(g) (1 + g sigmoid(-g))
    gate, up = s["x"].double().split(c["width"], dim=1)
    dy, sig = s["dy"].double(), torch.sigmoid(gate)
    dgate = dy * up * sig * (1 + gate * torch.sigmoid(-gate))
    return {"dx": torch.cat([dgate, dy * gate * sig], 1), "out": gate * sig * up if c["out"] else None}


# -------------------------------------------------------------------- work

def work(case):
    """Bytes and operations that a pass cannot do without: inputs read once, outputs written once."""
    c = case
    if c["op"] in ("product", "product8"):
        rows, n, k, E = c["rows"], c["n"], c["k"], c["experts"]
        used = E * (1 - (1 - 1 / E) ** rows)                       # experts that get a row, on average
        size = 2 if c["op"] == "product" else 1
        total = rows * k * size + used * n * k * size + rows * n * 2 + 4 * (E + 1)
        flops = 2 * rows * n * k
        if c["op"] == "product8":
            blocks = -(-k // _GROUP) * -(-n // _GROUP)
            total += 4 * (rows * -(-k // _GROUP) + used * blocks)
        if c["grad"]:
            total += rows * n * size + rows * k * 2                 # dy, dx
            flops *= 2
            if c["op"] == "product":
                total += E * n * k * size                           # dw
                flops += 2 * rows * n * k
            else:
                total += 4 * rows * -(-n // _GROUP)
        return {"bytes": int(total), "flops": flops}
    values = c["rows"] * c["width"]
    if c["op"] == "act":
        total = values * (4 if c["gated"] else 2) + values * (2 * c["out"] + c["codes"])
        if c["codes"]:
            total += 4 * c["rows"] * -(-c["width"] // _GROUP)
        return {"bytes": total, "flops": values * (8 if c["gated"] else 3)}
    return {"bytes": values * (10 + 2 * c["out"]), "flops": values * 14}
