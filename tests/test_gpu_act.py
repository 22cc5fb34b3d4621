"""GPU: the gated activation, its 8-bit output and its gradient against 64 bits.

Bounds.  In binary32 the sigmoid is an exponential (its exponent corrected), a
sum and a reciprocal, and three products follow: fewer than 16 roundings of at
most two units each, 2^-19 of the value.  Below the smallest normal number of
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
