"""hr_router_topk and its gradient on the GPU against the definitions in 64
bits: every layout's limits, odd numbers of experts, ties, masked and special
logits, strides, and what is left unpicked."""
import numpy as np
import pytest
import torch

from message_fp16_all_amd import hr
from _gpu import needs_gpu
from _rows import Maker, half_step, within

pytestmark = [pytest.mark.gpu, needs_gpu]

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# an exponent's argument, below 90 in magnitude for a weight that is not 0, is
# rounded to 24 bits: 90 x 2^-24 of the value, with the sum's roundings 2^-16
EXP = 2.0 ** -16
TINY = 2.0 ** -125


def reference(x, k, renormalize):
    """(ids, weights, p) of logits (CPU, any type) in 64 bits."""
    x = x.double().numpy()
    ok = x > -np.inf                                            # false for NaN
    top = np.where(ok, x, -np.inf).max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(ok, np.where(x == top, 1.0, np.exp(x - top)), 0.0)
    total = e.sum(1, keepdims=True)
    p = np.divide(e, total, out=np.zeros_like(e), where=total > 0)
    ids = np.full((len(x), k), -1)
    for i in range(len(x)):
        # sorted by value downward, index upward (-0 equals +0)
        order = sorted(np.flatnonzero(ok[i]), key=lambda c: (-x[i, c], c))[:k]
        ids[i, :len(order)] = order
    w = np.where(ids >= 0, np.take_along_axis(p, np.maximum(ids, 0), 1), 0.0)
    if renormalize:
        s = w.sum(1, keepdims=True)
        w = np.divide(w, s, out=np.zeros_like(w), where=s > 0)
    return torch.from_numpy(ids), torch.from_numpy(w), torch.from_numpy(p)


def grad_reference(g, ids, w, p, renormalize):
    """(dlogits, the magnitudes that go into it) in 64 bits."""
    there = ids >= 0
    g = torch.where(there, g.double(), 0.0)
    c, cs = (g * w).sum(1, keepdim=True), (g * w).abs().sum(1, keepdim=True)
    d, size = torch.zeros_like(p), torch.zeros_like(p)
    if not renormalize:
        d, size = -p * c, p * cs
    for j in range(ids.shape[1]):
        r = torch.nonzero(there[:, j])[:, 0]
        d[r, ids[r, j]] += w[r, j] * (g[r, j] - (c[r, 0] if renormalize else 0.0))
        size[r, ids[r, j]] += w[r, j] * (g[r, j].abs() + (cs[r, 0] if renormalize else 0.0))
    return d, size


def run(x, k, renormalize, what, stride=None, offset=0, in_place=False):
    tokens, experts = x.shape
    m = Maker(77)
    print(f"router {what}: {tokens}x{experts} k={k} {x.dtype} renormalize={renormalize}", flush=True)
    d = m.place(tokens, experts, x.dtype, stride, offset, x)
    w = torch.full((tokens, k), 9.0, device="cuda:0")
    ids = torch.full((tokens, k), 9, dtype=torch.int32, device="cuda:0")
    hr.router_topk(d, w, ids, renormalize=renormalize)
    torch.cuda.synchronize()
    iref, wref, p = reference(x, k, renormalize)
    assert torch.equal(ids.cpu().long(), iref), f"{what}: picks differ"
    within(w, wref, wref * EXP + TINY, f"{what}: weights")

    g = m.normal(tokens, k)
    g[iref < 0] = float("nan")                                  # what no pick has is not used
    dx = d if in_place else m.place(tokens, experts, x.dtype, stride, offset + 1)
    hr.router_topk_grad(g.cuda(), w, ids, dx, logits=None if renormalize else d, renormalize=renormalize)
    torch.cuda.synchronize()
    ref, size = grad_reference(g, iref, wref, p, renormalize)
    within(dx, ref, half_step(x.dtype, ref) * (1 + EXP) + size * 4 * EXP + TINY, f"{what}: dlogits")
    m.check_frames()


# both sides of every layout's limit in experts and picks
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("experts,k", [(1, 1), (2, 2), (7, 3), (8, 8), (9, 9), (60, 4), (64, 8), (64, 9), (65, 8),
                                       (128, 8), (128, 16), (128, 17), (129, 1), (160, 6), (255, 8), (256, 16),
                                       (256, 32), (257, 8), (384, 8), (512, 32), (513, 32), (1000, 10), (1024, 32)])
def test_layouts(dt, experts, k):
    m = Maker(experts + k)
    x = m.normal(37, experts, sigma=2.0, dtype=TYPES[dt])
    for renormalize in (False, True):
        run(x, k, renormalize, "layout")


@pytest.mark.parametrize("tokens", [0, 1, 2, 31, 32, 33, 4099])
def test_tokens(tokens):
    x = Maker(tokens).normal(tokens, 64, dtype=torch.bfloat16)
    if tokens == 0:
        w, ids = torch.empty(0, 4, device="cuda:0"), torch.empty(0, 4, dtype=torch.int32, device="cuda:0")
        hr.router_topk(x.cuda(), w, ids)
        hr.router_topk_grad(w, w, ids, x.cuda(), logits=x.cuda())
        return
    run(x, 4, True, "tokens")


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_ties_and_signed_zeros(dt, renormalize):
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-2, 3, (200, 96), generator=g).float()
    x = torch.where((x == 0) & (torch.rand(200, 96, generator=g) < 0.5), -0.0, x).to(TYPES[dt])
    x[0] = 0.0
    x[1] = -0.0
    x[2, ::2] = -0.0
    x[2, 1::2] = 0.0
    run(x, 9, renormalize, "ties")


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_masked_and_special(dt, renormalize):
    dtype = TYPES[dt]
    inf, nan, big = float("inf"), float("nan"), torch.finfo(dtype).max
    x = Maker(8).normal(12, 40, dtype=dtype)
    x[0] = -inf                                                 # nothing to pick
    x[1] = nan
    x[2, 3:] = -inf                                             # fewer than k
    x[3, ::2] = nan
    x[4] = -big                                                 # the lowest finite value is a value
    x[5, 7] = inf                                               # takes all
    x[6, 7] = x[6, 9] = inf                                     # share
    x[7] = inf
    x[8, 1:] = -big
    x[9] = torch.finfo(dtype).tiny / 8                          # subnormals
    x[9, 5] = torch.finfo(dtype).tiny / 4
    x[10, 39] = big
    x[11, :39] = -inf
    run(x, 6, renormalize, "special")
    x[:, 1], x[:, 30] = inf, big                                # the largest finite value beside an infinity
    run(x, 6, renormalize, "largest")


@pytest.mark.parametrize("dt,stride,offset", [("f16", 201, 1), ("bf16", 256, 3), ("f32", 199, 1), ("f32", 203, 2)])
def test_strides_and_in_place(dt, stride, offset):
    x = Maker(6).normal(50, 199, sigma=3.0, dtype=TYPES[dt])
    for renormalize in (False, True):
        run(x, 8, renormalize, "strides", stride, offset)
        run(x, 8, renormalize, "in place", stride, offset, in_place=True)


def test_far_apart_logits():
    """Weights down to nothing: exponents over the whole range of binary32."""
    x = -torch.linspace(0, 120, 64)[None].repeat(3, 1)
    run(x, 32, False, "far apart")
    run(x, 32, True, "far apart")


def test_foreign_ids_are_no_picks():
    x = Maker(2).normal(4, 16)
    ids = torch.tensor([[0, 99], [-5, 3], [16, 1 << 30], [2, 5]], dtype=torch.int32)
    w, g = torch.rand(4, 2), torch.rand(4, 2)
    clean = torch.where((ids >= 0) & (ids < 16), ids, -1).long()
    dx = torch.empty(4, 16, device="cuda:0")
    hr.router_topk_grad(g.cuda(), w.cuda(), ids.cuda(), dx, renormalize=True)
    ref, size = grad_reference(g, clean, torch.where(clean >= 0, w.double(), 0.0), torch.zeros(4, 16).double(), True)
    within(dx, ref, half_step(torch.float32, ref) + size * EXP, "dlogits")


def test_grad_against_differences():
    """Central differences of the weights in 64 bits, step 1e-5: their error,
    step^2 times a third derivative below 1, is far under the bound."""
    m = Maker(31)
    x, k, step = m.normal(3, 12), 4, 1e-5
    g = m.normal(3, k)
    for renormalize in (False, True):
        ids, wref, p = reference(x, k, renormalize)

        def loss(x):
            q = torch.softmax(x, 1).gather(1, ids)
            return (g.double() * (q / q.sum(1, keepdim=True) if renormalize else q)).sum()

        ref = torch.zeros(3, 12, dtype=torch.float64)
        for i in range(3):
            for j in range(12):
                e = torch.zeros(3, 12, dtype=torch.float64)
                e[i, j] = step
                ref[i, j] = (loss(x.double() + e) - loss(x.double() - e)) / (2 * step)
        w, di = torch.empty(3, k, device="cuda:0"), torch.empty(3, k, dtype=torch.int32, device="cuda:0")
        dx = torch.empty(3, 12, device="cuda:0")
        hr.router_topk(x.cuda(), w, di, renormalize=renormalize)
        hr.router_topk_grad(g.cuda(), w, di, dx, logits=x.cuda(), renormalize=renormalize)
        _, size = grad_reference(g, ids, wref, p, renormalize)
        within(dx, ref, size * 4 * EXP + 1e-8, "dlogits")


def test_stream_and_graph():
    m = Maker(1)
    x = m.normal(513, 256, dtype=torch.float16).cuda()
    w, ids = torch.empty(513, 8, device="cuda:0"), torch.empty(513, 8, dtype=torch.int32, device="cuda:0")
    g, dx = m.normal(513, 8).cuda(), torch.empty_like(x)

    def step(stream=None):
        hr.router_topk(x, w, ids, stream=stream)
        hr.router_topk_grad(g, w, ids, dx, logits=x, stream=stream)

    graph = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    s = torch.cuda.Stream()
    for k in range(3):
        x.copy_(m.normal(513, 256, dtype=torch.float16))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (w, ids, dx)]
        for again in (graph.replay, lambda: step(s)):
            for t in (w, ids, dx):
                t.zero_()
            torch.cuda.synchronize()
            again()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, (w, ids, dx)))


def test_binding_refusals():
    x = torch.zeros(4, 16, device="cuda:0")
    w, ids = torch.empty(4, 2, device="cuda:0"), torch.empty(4, 2, dtype=torch.int32, device="cuda:0")
    for bad, err in [(lambda: hr.router_topk(x.double(), w, ids), TypeError),
                     (lambda: hr.router_topk(x.cpu(), w, ids), TypeError),
                     (lambda: hr.router_topk(x, w.half(), ids), TypeError),
                     (lambda: hr.router_topk(x, w, ids.long()), TypeError),
                     (lambda: hr.router_topk(x, w[:3], ids), ValueError),
                     (lambda: hr.router_topk(x.t(), w, ids), ValueError),
                     (lambda: hr.router_topk(x[:, :1], w, ids), hr.HrError),
                     (lambda: hr.router_topk_grad(w, w, ids, x), hr.HrError),
                     (lambda: hr.router_topk_grad(w, w, ids, x, logits=x.half()), TypeError),
                     (lambda: hr.router_topk_grad(w, w, ids, x, logits=x[:3]), ValueError)]:
        with pytest.raises(err):
            bad()
    hr.router_topk(x, w, ids)
    assert ids.cpu().tolist() == [[0, 1]] * 4 and (w == 1 / 16).all()


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("experts", [32, 64, 200, 700])
def test_small_weights_are_exact_too(dt, experts):
    """Weights and gradients of logits up to 60 below the largest, relative to
    one another, so that the softmax's sum falls out of them.  The differences
    of these logits are exact in binary32.  An exponential is off by the unit in
    the last place of the instruction, 2^-23, one more rounding and 60 x 2^-28
    for ln 2, and every quotient or product by 2^-24: below 2^-21.  Two of them
    are compared, hence 2^-20."""
    g = torch.Generator().manual_seed(experts)
    x = -torch.randint(0, 60 * 64 + 1, (300, experts), generator=g) / 64.0
    x[torch.arange(300), torch.randint(0, experts, (300,), generator=g)] = 1.0
    x = x.to(TYPES[dt])
    d, k = x.cuda(), 32
    dw = torch.zeros(300, k)
    dw[:, 0] = 1.0
    xs = x.double()
    for renormalize in (False, True):
        w, ids = torch.empty(300, k, device="cuda:0"), torch.empty(300, k, dtype=torch.int32, device="cuda:0")
        print(f"small weights {dt} {experts} renormalize={renormalize}", flush=True)
        hr.router_topk(d, w, ids, renormalize=renormalize)
        torch.cuda.synchronize()
        v = xs.gather(1, ids.cpu().long())
        ref = torch.exp(v - v[:, :1])
        got = w.double().cpu()
        within(got / got[:, :1], ref, ref * 2.0 ** -20, "weights")
    if experts > k and dt == "f32":
        dx = torch.empty_like(d)
        hr.router_topk(d, w, ids)
        hr.router_topk_grad(dw.cuda(), w, ids, dx, logits=d)
        torch.cuda.synchronize()
        rest = torch.ones(300, experts, dtype=torch.bool).scatter_(1, ids.cpu().long(), False)
        got = dx.double().cpu()[rest].view(300, -1)
        v = xs[rest].view(300, -1)
        top, at = v.max(1, keepdim=True)
        ref = torch.exp(v - top)
        within(got / got.gather(1, at), ref, ref * 2.0 ** -20, "dlogits")
