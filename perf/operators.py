"""The operators around the combine, as cases to measure.

Three operators of a layer whose experts are spread over the ranks of an
all-reduce group:

* ``norm`` / ``norm_grad``: the fold of G contributions with the residual as
  its last operand, the root-mean-square norm of the sum, and its output in 16
  bits, in e4m3 with scales, or both; and the norm's gradient;
* ``router``: the k largest logits of every token with their softmax weights,
  and their gradient;
* ``experts``: tokens sorted by expert, gathered, and combined back with their
  weights, and the gradients.

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with the calls of ``message_fp16_all_amd.hr``.
"""
import functools
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_F8 = torch.float8_e4m3fn
_F8_MAX = 448.0
_F32_MIN = 2.0 ** -126
_EPS = 1e-6
_GROUP = 128
_MASKED = float("-inf")


def listed():
    return [
        # one decoded token of a two-rank group: the call's latency is all there is
        dict(name="norm 1x4096 G2", op="norm", dtype="f16", rows=1, hidden=4096, G=2, residual=True,
             weight="same", out=True, rstd=False, codes="none"),
        # a full decode batch of eight ranks, straight into an 8-bit product with one scale per 128 values
        dict(name="norm 64x6144 G8 e4m3", op="norm", dtype="bf16", rows=64, hidden=6144, G=8, residual=True,
             weight="f32", out=False, rstd=False, codes="group"),
        # a prefill chunk of eight ranks, with what a backward pass keeps: the largest fold
        dict(name="norm 2048x8192 G8", op="norm", dtype="f16", rows=2048, hidden=8192, G=8, residual=True,
             weight="same", out=True, rstd=True, codes="none"),
        # already summed activations of a ragged prefill batch, both outputs, one scale per token
        dict(name="norm 4999x5120 G1 e4m3", op="norm", dtype="bf16", rows=4999, hidden=5120, G=1, residual=True,
             weight="same", out=True, rstd=False, codes="row"),
        # training: the gradient of the norm over a chunk, joined by the residual stream's
        dict(name="norm_grad 2048x8192", op="norm_grad", dtype="bf16", rows=2048, hidden=8192, residual=True,
             weight="f32"),
        # the same of an odd number of short rows: the heads of a query, normed one by one
        dict(name="norm_grad 65537x128", op="norm_grad", dtype="f16", rows=65537, hidden=128, residual=False,
             weight="same"),
        # a decode batch choosing its experts
        dict(name="router 64x128 k8", op="router", dtype="f32", tokens=64, experts=128, k=8, renormalize=True,
             masked=False, grad=False),
        # a training batch with masked experts, both directions, weights not renormalised
        dict(name="router 32768x256 k8 grad", op="router", dtype="bf16", tokens=32768, experts=256, k=8,
             renormalize=False, masked=True, grad=True),
        # one decoded token and its experts
        dict(name="experts 1x4096 k8", op="experts", dtype="f16", tokens=1, hidden=4096, experts=128, first=0,
             local=128, k=8, pad=1, codes=False, grad=False),
        # a decode batch on the rank that holds a quarter of the experts, in 8 bits, segments padded to 16 rows
        dict(name="experts 64x5120 k6 e4m3", op="experts", dtype="bf16", tokens=64, hidden=5120, experts=64, first=16,
             local=16, k=6, pad=16, codes=True, grad=False),
        # an odd prefill batch over every expert
        dict(name="experts 8191x4096 k8", op="experts", dtype="bf16", tokens=8191, hidden=4096, experts=128, first=0,
             local=128, k=8, pad=1, codes=False, grad=False),
        # a training step: there, back, and both gradients, segments padded to a product's tile
        dict(name="experts 4096x8192 k4 grad", op="experts", dtype="f16", tokens=4096, hidden=8192, experts=32,
             first=0, local=32, k=4, pad=128, codes=False, grad=True),
    ]


def _spread(rng, low, high):
    """A whole number spread over the logarithm: a power of two or an odd one."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    if rng.random() < 0.4:
        return max(low, 1 << int(math.log2(v)))
    return min(high, int(v) | 1)


def _width(rng):
    """A row length: mostly an odd multiple of 64 or a power of two, sometimes odd itself."""
    if rng.random() < 0.25:
        return _spread(rng, 64, 16384)
    return rng.choice([1 << rng.randint(6, 14), 64 * _spread(rng, 1, 255)])


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "router", "experts", "experts"])
    most = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    while True:
        if op == "norm":
            out = rng.random() < 0.7
            case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), rows=_spread(rng, 1, 65536), hidden=_width(rng),
                        G=rng.choice([1, 1, 2, 3, 4, 5, 8, 16]), residual=rng.random() < 0.8,
                        weight=rng.choice(["same", "f32", "none"]), out=out, rstd=rng.random() < 0.3,
                        codes=rng.choice(["none", "row", "group"]) if out else rng.choice(["row", "group"]))
        elif op == "norm_grad":
            case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), rows=_spread(rng, 1, 131072), hidden=_width(rng),
                        residual=rng.random() < 0.5, weight=rng.choice(["same", "f32"]))
        elif op == "router":
            experts = rng.choice([8, 16, 32, 60, 64, 96, 128, 160, 256, 384, 512])
            case = dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), tokens=_spread(rng, 1, 32768),
                        experts=experts, k=rng.randint(1, min(10, experts)), renormalize=rng.random() < 0.5,
                        masked=rng.random() < 0.5, grad=rng.random() < 0.5)
        else:
            experts = rng.choice([8, 16, 32, 60, 64, 96, 128, 160, 256, 384, 512])
            parts = rng.choice([1, 1, 2, 4])
            case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), tokens=_spread(rng, 1, 32768), hidden=_width(rng),
                        experts=experts, first=experts // parts * rng.randrange(parts), local=experts // parts,
                        k=rng.randint(1, min(8, experts)), pad=rng.choice([1, 1, 16, 64, 128]),
                        codes=rng.random() < 0.3, grad=rng.random() < 0.4)
            if _rows(case) * case["hidden"] > 2 * 8192 * 8 * 4096:
                continue
        if work(case)["bytes"] <= most:
            return case


def _rows(case):
    """Rows that the sorted tokens take at most: every segment that holds one is rounded up."""
    slots = case["tokens"] * case["k"]
    return slots + min(case["local"], slots) * (case["pad"] - 1)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    {"norm": _prepare_norm, "norm_grad": _prepare_norm_grad, "router": _prepare_router,
     "experts": _prepare_experts}[case["op"]](case, g, state)
    return state


def _normal(g, *shape, sigma=1.0, dtype=torch.float32):
    x = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)
    return x.mul_(sigma) if sigma != 1.0 else x


def _weight(case, g):
    if case["weight"] == "none":
        return None
    w = _normal(g, case["hidden"], sigma=0.1) + 1.0
    return w if case["weight"] == "f32" else w.to(_TYPES[case["dtype"]])


def _prepare_norm(case, g, s):
    rows, hidden, dt = case["rows"], case["hidden"], _TYPES[case["dtype"]]
    # partial sums of a layer, and a residual stream with a few outlying channels
    s["x"] = [_normal(g, rows, hidden, sigma=0.5, dtype=dt) for _ in range(case["G"])]
    s["residual"] = _normal(g, rows, hidden, dtype=dt) if case["residual"] else None
    if case["residual"]:
        s["residual"][:, ::97] *= 8
    s["weight"] = _weight(case, g)
    new = functools.partial(torch.empty, device="cuda")
    s["h"] = new(rows, hidden, dtype=dt) if case["residual"] else None
    s["out"] = new(rows, hidden, dtype=dt) if case["out"] else None
    s["rstd"] = new(rows) if case["rstd"] else None
    s["group"] = _GROUP if case["codes"] == "group" else 0
    groups = -(-hidden // _GROUP) if s["group"] else 1
    s["codes"] = new(rows, hidden, dtype=_F8) if case["codes"] != "none" else None
    s["scales"] = new(rows, groups) if case["codes"] != "none" else None


def _prepare_norm_grad(case, g, s):
    rows, hidden, dt = case["rows"], case["hidden"], _TYPES[case["dtype"]]
    s["h"] = _normal(g, rows, hidden, sigma=2.0, dtype=dt)
    s["dy"] = _normal(g, rows, hidden, sigma=0.1, dtype=dt)
    s["dres"] = _normal(g, rows, hidden, sigma=0.1, dtype=dt) if case["residual"] else None
    s["weight"] = _weight(case, g)
    s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + _EPS)
    s["dx"] = torch.empty_like(s["h"])
    s["dweight"] = torch.empty(hidden, device="cuda")


def _prepare_router(case, g, s):
    T, E, k = case["tokens"], case["experts"], case["k"]
    # some experts are more liked than others
    x = _normal(g, T, E) + _normal(g, E)
    if case["masked"]:
        x[torch.rand(T, E, generator=g, device="cuda") < 0.1] = _MASKED
        x[torch.rand(T, generator=g, device="cuda") < 0.02] = _MASKED     # padding tokens choose nothing
    s["logits"] = x.to(_TYPES[case["dtype"]])
    s["weights"] = torch.empty(T, k, device="cuda")
    s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
    if case["grad"]:
        s["dweights"] = _normal(g, T, k)
        s["dlogits"] = torch.empty_like(s["logits"])


def _prepare_experts(case, g, s):
    T, H, E, k, dt = case["tokens"], case["hidden"], case["experts"], case["k"], _TYPES[case["dtype"]]
    liked = _normal(g, T, E) + _normal(g, E)
    ids = torch.sort(liked, dim=1, descending=True)[1][:, :k].to(torch.int32)
    if T > 16:
        ids[torch.rand(T, generator=g, device="cuda") < 0.02] = -1        # padding tokens
    s["ids"] = ids.contiguous()
    w = torch.rand(T, k, generator=g, device="cuda") + 0.05
    s["weights"] = w / w.sum(1, keepdim=True)
    rows = _rows(case)
    zeros = functools.partial(torch.zeros, device="cuda")
    if case["codes"]:
        s["x"] = _normal(g, T, H, sigma=100.0).clamp_(-_F8_MAX, _F8_MAX).to(_F8)
        s["scales"] = torch.rand(T, -(-H // _GROUP), generator=g, device="cuda") + 0.01
        s["sorted_scales"] = zeros(rows, s["scales"].shape[1])
    else:
        s["x"] = _normal(g, T, H, dtype=dt)
    s["offsets"] = zeros(case["local"] + 1, dtype=torch.int32)
    s["order"] = zeros(rows, dtype=torch.int32)
    s["pos"] = zeros(T, k, dtype=torch.int32)
    s["sorted"] = zeros(rows, H, dtype=s["x"].dtype)
    # what the experts answer with, and the rows that a gradient comes back in
    s["z"] = _normal(g, rows, H, dtype=dt)
    s["out"] = zeros(T, H, dtype=dt)
    if case["grad"]:
        s["dout"] = _normal(g, T, H, sigma=0.1, dtype=dt)
        s["dsorted"] = _normal(g, rows, H, sigma=0.1, dtype=dt)
        s["dz"] = zeros(rows, H, dtype=dt)
        s["dweights"] = zeros(T, k)
        s["dx"] = zeros(T, H, dtype=dt)


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


def _own_norm(s):
    _hr.reduce_rmsnorm(s["x"], s["out"], residual=s["residual"], residual_out=s["h"], weight=s["weight"], eps=_EPS,
                       out8=s["codes"], scales=s["scales"], group=s["group"], rstd=s["rstd"])
    return {"h": s["h"], "y": s["out"], "codes": s["codes"], "scales": s["scales"], "rstd": s["rstd"]}


def _own_norm_grad(s):
    _hr.rmsnorm_grad(s["dy"], s["h"], s["rstd"], s["dx"], weight=s["weight"], dresidual=s["dres"],
                     dweight=s["dweight"])
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _own_router(s):
    again = s["case"]["renormalize"]
    _hr.router_topk(s["logits"], s["weights"], s["ids"], renormalize=again)
    out = {"weights": s["weights"], "ids": s["ids"]}
    if s["case"]["grad"]:
        _hr.router_topk_grad(s["dweights"], s["weights"], s["ids"], s["dlogits"], logits=s["logits"],
                             renormalize=again)
        out["dlogits"] = s["dlogits"]
    return out


def _own_experts(s):
    c = s["case"]
    _hr.experts_sort(s["ids"], s["offsets"], s["order"], s["pos"], first=c["first"], pad=c["pad"])
    _hr.experts_gather(s["x"], s["pos"], s["sorted"], offsets=s["offsets"], order=s["order"],
                       scales=s.get("scales"), scales_out=s.get("sorted_scales"))
    _hr.experts_combine(s["z"], s["pos"], s["out"], weights=s["weights"])
    if c["grad"]:
        _hr.experts_combine_grad(s["dout"], s["z"], s["pos"], s["weights"], s["dz"], s["dweights"],
                                 offsets=s["offsets"], order=s["order"])
        _hr.experts_combine(s["dsorted"], s["pos"], s["dx"])
    return _experts_out(s)


def _experts_out(s):
    names = ["offsets", "order", "pos", "sorted", "out"]
    names += ["sorted_scales"] if s["case"]["codes"] else []
    names += ["dz", "dweights", "dx"] if s["case"]["grad"] else []
    return {n: s[n] for n in names}


_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "router": _own_router, "experts": _own_experts}


# ------------------------------------------------------------- plain forms

def _add(a, b):
    """One add of the combine: 16-bit values, one rounding to their type."""
    return (a.float() + b.float()).to(a.dtype)


def _plain_norm(s):
    c = s["case"]
    h = functools.reduce(_add, s["x"] + ([s["residual"]] if c["residual"] else []))
    f = h.float()
    rstd = 1.0 / torch.sqrt(f.square().mean(1) + _EPS)
    y = f * rstd[:, None]
    if s["weight"] is not None:
        y = y * s["weight"].float()
    codes = scales = None
    if c["codes"] == "row":
        scales = (y.abs().amax(1, keepdim=True) / _F8_MAX).clamp_min(_F32_MIN)
        codes = (y / scales).to(_F8)
    elif c["codes"] == "group":
        rows, hidden = y.shape
        groups = s["scales"].shape[1]
        whole = torch.nn.functional.pad(y, (0, groups * _GROUP - hidden)).view(rows, groups, _GROUP)
        scales = (whole.abs().amax(2) / _F8_MAX).clamp_min(_F32_MIN)
        codes = (whole / scales[:, :, None]).view(rows, -1)[:, :hidden].contiguous().to(_F8)
    return {"h": h if c["residual"] else None, "y": y.to(h.dtype) if c["out"] else None, "codes": codes,
            "scales": scales, "rstd": rstd if c["rstd"] else None}


def _plain_norm_grad(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    unit = s["h"].float() * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - unit * (g * unit).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * unit).sum(0)}


def _plain_router(s):
    c = s["case"]
    x = s["logits"].float()
    there = x > _MASKED
    top = x.amax(1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    e = torch.where(there, torch.exp(x - top), 0.0)
    p = e / e.sum(1, keepdim=True).clamp_min(_F32_MIN)
    at = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :c["k"]]
    picked = there.gather(1, at)
    w = torch.where(picked, p.gather(1, at), 0.0)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True).clamp_min(_F32_MIN)
    out = {"weights": w, "ids": torch.where(picked, at, -1).to(torch.int32)}
    if c["grad"]:
        g = torch.where(picked, s["dweights"], 0.0)
        mean = (g * w).sum(1, keepdim=True)
        if c["renormalize"]:
            d = torch.zeros_like(x).scatter_(1, at, w * (g - mean))
        else:
            d = p * (torch.zeros_like(x).scatter_(1, at, g) - mean)
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _plain_experts(s):
    c = s["case"]
    T, k, E, pad, rows = c["tokens"], c["k"], c["local"], c["pad"], s["order"].numel()
    dev = s["ids"].device
    e = s["ids"].reshape(-1) - c["first"]
    e = torch.where((e >= 0) & (e < E), e, E).long()
    slots = torch.sort(e, stable=True)[1]
    count = torch.zeros(E + 1, dtype=torch.int64, device=dev).scatter_add_(0, e, torch.ones_like(e))
    ends = torch.cumsum((count[:E] + pad - 1) // pad * pad, 0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    # the place of the i-th slot in sorted order: its segment's start and its number in it
    of = e[slots]
    before = torch.cumsum(count, 0) - count
    place = offsets[of] + torch.arange(T * k, device=dev) - before[of]
    place = torch.where(of < E, place, rows)
    order = torch.full((rows + 1,), -1, dtype=torch.int64, device=dev).scatter_(0, place, slots)[:rows]
    pos = torch.empty_like(e).scatter_(0, slots, torch.where(of < E, place, -1)).view(T, k)
    here = order >= 0
    token = order.clamp_min(0) // k
    s_out = {"offsets": offsets.to(torch.int32), "order": torch.where(here, order, -1).to(torch.int32),
             "pos": pos.to(torch.int32)}
    raw = s["x"].view(torch.uint8) if c["codes"] else s["x"]
    out = (raw[token] * here[:, None]).view(s["x"].dtype)
    s_out["sorted"] = out
    if c["codes"]:
        s_out["sorted_scales"] = s["scales"][token] * here[:, None]
    there = pos >= 0
    at = pos.clamp_min(0)
    w = s["weights"] * there

    def back(z, w):
        return functools.reduce(torch.add, [z[at[:, j]].float() * w[:, j, None] for j in range(k)])

    s_out["out"] = back(s["z"], w).to(s["z"].dtype)
    if c["grad"]:
        dout = s["dout"].float()
        flat = w.reshape(-1)[order.clamp_min(0)] * here
        s_out["dz"] = (s["dout"][token].float() * flat[:, None]).to(s["z"].dtype)
        dots = [(dout * s["z"][at[:, j]].float()).sum(1) for j in range(k)]
        s_out["dweights"] = torch.stack(dots, 1) * there
        s_out["dx"] = back(s["dsorted"], there.float()).to(s["z"].dtype)
    return s_out


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "router": _plain_router, "experts": _plain_experts}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The same from the definitions in 64 bits, before the last rounding to a type."""
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "router": _exact_router,
            "experts": _exact_experts}[case["op"]](case, s)


def _exact_norm(c, s):
    terms = [x.double() for x in s["x"]]
    if c["residual"]:
        terms.append(s["residual"].double())
    total = terms[0]
    for t in terms[1:]:
        # the combine's own definition: every add ends in the operands' type
        total = (total + t).to(_TYPES[c["dtype"]]).double()
    power = (total * total).sum(1) / c["hidden"]
    rstd = (power + _EPS) ** -0.5
    y = total * rstd[:, None]
    if s["weight"] is not None:
        y *= s["weight"].double()
    codes = scales = None
    if c["codes"] != "none":
        width = _GROUP if c["codes"] == "group" else c["hidden"]
        largest = [part.abs().max(dim=1).values for part in y.split(width, dim=1)]
        scales = torch.stack(largest, 1) / _F8_MAX
        codes = torch.cat([part / scales[:, i:i + 1] for i, part in enumerate(y.split(width, dim=1))], 1)
    return {"h": total if c["residual"] else None, "y": y if c["out"] else None, "codes": codes, "scales": scales,
            "rstd": rstd if c["rstd"] else None}


def _exact_norm_grad(c, s):
    # the derivative of sum(dy * y) + sum(dres * h), y = w h / sqrt(mean(h^2) + eps), with rstd as it was kept
    h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()
    wdy = dy * s["weight"].double()
    along = (wdy * h).sum(1) * r ** 3 / c["hidden"]
    dx = wdy * r[:, None] - h * along[:, None]
    if s["dres"] is not None:
        dx += s["dres"].double()
    return {"dx": dx, "dweight": (dy * h * r[:, None]).sum(0)}


def _exact_router(c, s):
    x = s["logits"].double()
    T, E = x.shape
    p = torch.nan_to_num(torch.softmax(x, 1))                  # a row with nothing in it has no weights
    # by logit downward, then by index upward: the rank of each expert is how many come before it
    left, ids, w = x.clone(), [], []
    rows = torch.arange(T, device=x.device)
    for _ in range(c["k"]):
        best = left.max(1, keepdim=True).values
        at = torch.where(left == best, torch.arange(E, device=x.device), E).min(1).values
        ids.append(torch.where(best[:, 0] > _MASKED, at, -1))
        w.append(torch.where(best[:, 0] > _MASKED, p[rows, at], 0.0))
        left[rows, at] = _MASKED
    ids, w = torch.stack(ids, 1), torch.stack(w, 1)
    if c["renormalize"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    out = {"weights": w, "ids": None}
    if c["grad"]:
        g = torch.zeros(T, E + 1, dtype=torch.float64, device=x.device)
        g.scatter_(1, torch.where(ids >= 0, ids, E), s["dweights"].double())
        g = g[:, :E]
        chosen = torch.zeros(T, E + 1, dtype=torch.bool, device=x.device)
        chosen.scatter_(1, torch.where(ids >= 0, ids, E), True)
        q = p
        if c["renormalize"]:
            q = torch.where(chosen[:, :E], p, 0.0)
            q = torch.nan_to_num(q / q.sum(1, keepdim=True))
        out["dlogits"] = q * (g - (q * g).sum(1, keepdim=True))
    return out


def _exact_experts(c, s):
    T, k = c["tokens"], c["k"]
    ids = s["ids"].cpu().reshape(-1).tolist()
    where, segment = [-1] * (T * k), [[] for _ in range(c["local"])]
    for slot, e in enumerate(ids):
        if 0 <= e - c["first"] < c["local"]:
            segment[e - c["first"]].append(slot)
    row = 0
    for slots in segment:
        for i, slot in enumerate(slots):
            where[slot] = row + i
        row += -(-len(slots) // c["pad"]) * c["pad"]
    pos = torch.tensor(where, device="cuda").view(T, k)
    out = {n: None for n in ("offsets", "order", "pos", "sorted", "sorted_scales", "dz", "dweights", "dx")}
    y = torch.zeros(T, c["hidden"], dtype=torch.float64, device="cuda")
    dx = torch.zeros_like(y)
    dots = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    if c["grad"]:
        dz = torch.zeros(s["z"].shape, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        p = pos[t, j]
        z, w = s["z"][p].double(), s["weights"][t, j].double()
        y[t] += z * w[:, None]
        if c["grad"]:
            dy = s["dout"][t].double()
            dots[t, j] = (dy * z).sum(1)
            dz[p] = dy * w[:, None]
            dx[t] += s["dsorted"][p].double()
    out["out"] = y
    if c["grad"]:
        out.update(dz=dz, dweights=dots, dx=dx)
    return out


# -------------------------------------------------------------------- work

def work(case):
    """Bytes and operations that a pass cannot do without: inputs read once, outputs written once."""
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["hidden"]
        groups = -(-c["hidden"] // _GROUP) if c["codes"] == "group" else 1
        reads = n * 2 * (c["G"] + c["residual"]) + c["hidden"] * {"same": 2, "f32": 4, "none": 0}[c["weight"]]
        writes = n * 2 * (c["residual"] + c["out"]) + 4 * c["rows"] * c["rstd"]
        if c["codes"] != "none":
            writes += n + 4 * c["rows"] * groups
        return {"bytes": reads + writes, "flops": n * (c["G"] + 4)}
    if c["op"] == "norm_grad":
        n = c["rows"] * c["hidden"]
        small = 4 * c["rows"] + c["hidden"] * (4 + {"same": 2, "f32": 4}[c["weight"]])
        return {"bytes": n * 2 * (3 + c["residual"]) + small, "flops": n * 10}
    if c["op"] == "router":
        T, E, k = c["tokens"], c["experts"], c["k"]
        size = 4 if c["dtype"] == "f32" else 2
        reads = T * E * size + (4 * T * k if c["grad"] else 0)
        writes = 8 * T * k + (T * E * size if c["grad"] else 0)
        return {"bytes": reads + writes, "flops": T * E * (6 if c["grad"] else 3)}
    T, H, k = c["tokens"], c["hidden"], c["k"]
    # the share of the slots that this rank's experts take, as they are drawn here
    taken = T * k * c["local"] // c["experts"]
    size = 1 if c["codes"] else 2
    total = 4 * (2 * T * k + c["local"] + 1 + _rows(c))                  # ids, pos, offsets, order
    total += (T + taken) * H * size + 4 * T * k                          # gather, weights
    if c["codes"]:
        total += 4 * (T + taken) * -(-H // _GROUP)
    total += (taken + T) * H * 2                                         # combine
    flops = 2 * taken * H
    if c["grad"]:
        total += (T + 2 * taken) * H * 2 + 4 * T * k                     # dout, z again with it, dz
        total += (taken + T) * H * 2                                     # dsorted, dx
        flops += 4 * taken * H
    return {"bytes": total, "flops": flops}
