"""GPU: the gated activation, its 8-bit output and its gradient against 64 bits.

Bounds.  In binary32 the sigmoid is an exponential (its exponent corrected but
for what binary32 leaves out of log2(e), 1.93e-8 * 87 * ln 2 = 1.17e-6 below a
gate of 87), a sum and a reciprocal, and three products follow: six roundings
of at most a unit of 2^-23 each, 7.2e-7; together below 2^-19 of the value.  Below the smallest normal number of
binary32 a product is off by half a subnormal step, times at most 2^6 (the
gate) where it is multiplied on; half_step of the output covers float16, and
2^-142 bfloat16.  dgate has a sum, 1 + gate (1 - s), that can cancel: its terms
are bounded by dy * up * s * (1 + |gate| (1 - s)).  A code is the quotient of
the unrounded y by its scale, each off by that much, rounded by half a step.
"""
import pytest
import torch

from _gpu import needs_gpu
from _products import F8
from _rows import TYPES, Maker, half_step, within
from message_fp16_all_amd import hr

pytestmark = [pytest.mark.gpu, needs_gpu]
DEV = "cuda:0"
F32 = 2.0 ** -19
SMALL = 2.0 ** -142

# (rows, width)
SHAPES = [(1, 1), (3, 7), (2, 8), (5, 9), (4, 31), (7, 64), (3, 100), (9, 128), (2, 129), (17, 136), (5, 512), (3, 520),
          (2, 1001), (6, 2048), (2, 2056), (1, 10240)]


def gates(m, rows, width, dt, sigma=3.0):
    x = m.normal(rows, 2 * width, sigma=sigma, dtype=dt)
    flat = x.view(-1)
    if flat.numel() > 64:                                        # far from zero, both signs; zeros
        far = torch.tensor([0.0, -0.0, 20.0, -20.0, 44.0, -44.5, -60.0, 80.0, -80.0, -87.0, -90.0, -100.0, 100.0, -110.0])
        flat[torch.arange(far.numel()) * 4 + 3] = far.to(dt)
    return x


def act_ref(x, width):
    gate, up = x[:, :width].double(), x[:, width:].double()
    return gate * torch.sigmoid(gate) * up


def tol_of(dt, ref):
    return half_step(dt, ref) + ref.abs() * F32 + SMALL


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,width", SHAPES)
def test_act(name, rows, width):
    dt = TYPES[name]
    m = Maker(rows * 100 + width)
    x = gates(m, rows, width, dt)
    out = m.place(rows, width, dt, stride=width + 3, offset=1)
    hr.experts_act(m.place(rows, 2 * width, dt, stride=2 * width + 5, offset=3, values=x), out)
    ref = act_ref(x, width)
    within(out, ref, tol_of(dt, ref), "out")
    m.check_frames()


def check_codes(codes, scales, y, group, what):
    """codes * scale is y, and the scale y's largest value over 448, in each group."""
    codes, scales = codes.cpu().double(), scales.cpu().double()
    for g in range(scales.shape[1]):
        part = y[:, g * group:(g + 1) * group]
        top = part.abs().amax(1)
        want = torch.clamp(top / 448.0, min=2.0 ** -126)
        within(scales[:, g], want, want * (F32 + 2.0 ** -22), f"{what}: scales of group {g}")
        q = part / want[:, None]
        # half a step of e4m3 (2^-4 of the value, 2^-10 below its normal range)
        tol = torch.clamp(q.abs() * 2.0 ** -4, min=2.0 ** -10) + q.abs() * 2 ** -17
        within(codes[:, g * group:(g + 1) * group], q, tol, f"{what}: codes of group {g}")


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_codes(name, group, gated, rows, width):
    dt = TYPES[name]
    m = Maker(rows * 100 + width + group)
    x = m.normal(rows, width * (2 if gated else 1), sigma=2.0, dtype=dt)
    x[0] = 0.0                                                   # the smallest scale
    codes = torch.full((rows + 1, width + 3), 7.0).to(F8).to(DEV)
    scales = m.place(rows, -(-width // group), torch.float32, stride=-(-width // group) + 2)
    out = m.place(rows, width, dt)
    hr.experts_act(x.to(DEV), out, gated=gated, out8=codes[:rows, 1:width + 1], scales=scales, group=group)
    y = act_ref(x, width) if gated else x.double()
    check_codes(codes[:rows, 1:width + 1], scales, y, group, "act")
    within(out, y, tol_of(dt, y), "out")
    assert (codes[rows].float() == 7).all() and (codes[:, 0].float() == 7).all() and (codes[:, width + 1:].float() == 7).all()
    m.check_frames()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("again,same", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_act_grad(name, again, same, rows, width):
    dt = TYPES[name]
    m = Maker(rows * 100 + width + 1)
    x = gates(m, rows, width, dt)
    dy = m.normal(rows, width, dtype=dt)
    dx = m.place(rows, 2 * width, dt, stride=2 * width + 1, offset=1)
    if same:
        dx.copy_(x)
    out = m.place(rows, width, dt) if again else None
    hr.experts_act_grad(dy.to(DEV), dx if same else x.to(DEV), dx, out=out)
    gate, up, d = x[:, :width].double(), x[:, width:].double(), dy.double()
    s, rest = torch.sigmoid(gate), torch.sigmoid(-gate)
    dgate, dup = d * up * s * (1 + gate * rest), d * gate * s
    mag = (d * up * s).abs() * (1 + gate.abs() * rest)
    within(dx[:, :width], dgate, half_step(dt, dgate) + mag * F32 + SMALL, "dgate")
    within(dx[:, width:], dup, tol_of(dt, dup), "dup")
    if again:
        ref = act_ref(x, width)
        within(out, ref, tol_of(dt, ref), "out")
    m.check_frames()


@pytest.mark.parametrize("used", [0, 1, 5, 9, 12])
def test_rows_past_the_last_segment(used):
    m = Maker(used)
    dt, rows, width = torch.bfloat16, 9, 264
    at = torch.tensor([0, used // 2, used], dtype=torch.int32, device=DEV)
    x, dy = m.normal(rows, 2 * width, dtype=dt), m.normal(rows, width, dtype=dt)
    out, dx = m.place(rows, width, dt), m.place(rows, 2 * width, dt)
    scales, codes = m.place(rows, 3, torch.float32), torch.full((rows, width), 7.0).to(F8).to(DEV)
    hr.experts_act(x.to(DEV), out, offsets=at, out8=codes, scales=scales)
    hr.experts_act_grad(dy.to(DEV), x.to(DEV), dx, offsets=at)
    n = min(used, rows)
    ref = act_ref(x, width)
    within(out[:n], ref[:n], tol_of(dt, ref)[:n], "out")
    for t in (out, dx, scales, codes):
        assert (t[n:].float() == 7).all()
    if n:
        check_codes(codes[:n], scales[:n], ref[:n], 128, "act")
        assert not (dx[:n].float() == 7).all()


def test_not_finite():
    """NaN and infinities stay in their values (and their group's scale)."""
    x = torch.ones(4, 512, dtype=torch.float16)
    x[0, 3], x[1, 200], x[2, 256 + 40], x[3, 10] = float("nan"), float("inf"), float("nan"), -float("inf")
    out = torch.empty(4, 256, dtype=torch.float16, device=DEV)
    codes, scales = torch.empty(4, 256, dtype=F8, device=DEV), torch.empty(4, 2, device=DEV)
    hr.experts_act(x.to(DEV), out, out8=codes, scales=scales)
    bad = torch.zeros(4, 256, dtype=torch.bool)
    bad[0, 3] = bad[2, 40] = bad[3, 10] = True
    got, s = out.cpu(), scales.cpu()
    assert torch.equal(torch.isnan(got), bad) and got[1, 200] == float("inf")
    assert torch.isfinite(got[~bad]).sum() == (~bad).sum() - 1
    assert torch.equal(torch.isnan(s), torch.tensor([[True, False], [False, False], [True, False], [True, False]]))
    assert s[1, 1] == float("inf")
    dx = torch.empty(4, 512, dtype=torch.float16, device=DEV)
    hr.experts_act_grad(torch.ones(4, 256, dtype=torch.float16, device=DEV), x.to(DEV), dx)
    d = dx.cpu()
    assert torch.isfinite(d).sum() >= d.numel() - 8


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 40, generator=g).double()
    dy = torch.randn(3, 20, generator=g).half()
    h = x.half()
    dx = torch.empty(3, 40, dtype=torch.float16, device=DEV)
    hr.experts_act_grad(dy.to(DEV), h.to(DEV), dx)
    step = 1e-6
    for r in range(3):
        for c in range(40):
            up, down = h.double().clone(), h.double().clone()
            up[r, c] += step
            down[r, c] -= step
            slope = float(((act_ref(up, 20) - act_ref(down, 20)) * dy.double()).sum()) / (2 * step)
            # (a difference's own error: 1e-9 of values below 2^5)
            assert abs(float(dx[r, c]) - slope) <= abs(slope) * 2 ** -11 + 2 ** -24 + 1e-7


def test_graph():
    m, width = Maker(2), 1032
    x = torch.empty(70, 2 * width, dtype=torch.float16, device=DEV)
    out, again = torch.empty(70, width, dtype=torch.float16, device=DEV), torch.empty(70, width, dtype=torch.float16, device=DEV)
    codes, scales = torch.empty(70, width, dtype=F8, device=DEV), torch.empty(70, 9, device=DEV)
    hr.experts_act(x, out, out8=codes, scales=scales)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hr.experts_act(x, out, out8=codes, scales=scales)
    for _ in range(3):
        v = m.normal(70, 2 * width, sigma=2.0, dtype=torch.float16)
        x.copy_(v)
        graph.replay()
        hr.experts_act(x, again)
        torch.cuda.synchronize()
        assert torch.equal(out, again)
        check_codes(codes, scales, act_ref(v, width), 128, "act")


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,width", [(4096, 64), (2048, 504), (512, 2048)])
def test_a_value_does_not_depend_on_its_neighbours(name, rows, width):
    """Gates far from zero take another way to the sigmoid; the others' results have the same bits beside them."""
    dt = TYPES[name]
    m = Maker(rows + width)
    x, dy = m.normal(rows, 2 * width, sigma=20.0, dtype=dt).clamp(-80, 80).to(DEV), m.normal(rows, width, dtype=dt).to(DEV)
    far = x.clone()
    apart = torch.arange(rows * width, device=DEV).view(rows, width) % 31 == 0
    for value in (-100.0, 100.0, float("nan")):
        far[:, :width][apart] = value
        got = [[torch.zeros(rows, w, dtype=dt, device=DEV) for w in (width, 2 * width)] for _ in range(2)]
        for (out, dx), v in zip(got, (x, far)):
            hr.experts_act(v, out)
            hr.experts_act_grad(dy, v, dx)
        for a, b in zip(*got):
            a, b = a.view(rows, -1, width), b.view(rows, -1, width)
            assert torch.equal(a.movedim(1, 0)[:, ~apart], b.movedim(1, 0)[:, ~apart])
