"""GPU: the activation's calls of many values, which give a lane two rows and go past
the caches: bit for bit what the same rows give in small calls, which other tests
hold to 64 bits; rows past the last segment, and what lies between rows, left alone."""
import pytest
import torch

from _gpu import needs_gpu
from _products import F8
from _rows import TYPES
from message_fp16_all_amd import hr

pytestmark = [pytest.mark.gpu, needs_gpu]
DEV = "cuda:0"
STREAM = 1 << 27                                                 # bytes that such a call moves at least
# every number of lanes to a row, whole units and not
WIDTHS = [120, 127, 129, 264, 511, 520, 2048, 2049]


def lanes_of(width):
    return 16 if width <= 128 else 64 if width <= 512 else 256


def rows_of(width, per_value):
    """An odd number of rows, past the limit, whose last workgroup is not full."""
    high = 2 * 256 // lanes_of(width)
    rows = STREAM // (per_value * width) // high * high + 3 * high + 1
    assert rows * width * per_value >= STREAM and rows % 2 == 1
    return rows


def used_of(rows, width):
    """(how many rows in use): all; and an end after a lane's first row and before its second."""
    pair = 256 // lanes_of(width)
    end = rows // (2 * pair) * (2 * pair) - 2 * pair + (pair + 1) // 2
    return rows, end


def normal(g, *shape, dt):
    return torch.empty(*shape, dtype=dt, device=DEV).normal_(0.0, 2.0, generator=g)


def place(rows, width, dt, extra, offset, fill):
    """Rows apart inside a buffer that holds ``fill``: (buffer, rows)."""
    buf = torch.full((offset + rows * (width + extra),), fill, dtype=torch.uint8 if dt is F8 else torch.int16, device=DEV)
    if dt is torch.float32:
        buf = torch.full((offset + rows * (width + extra),), float(fill), device=DEV)
    view = buf.as_strided((rows, width), (width + extra, 1), offset)
    return buf, view if dt is torch.float32 else view.view(dt)


def raw(t):
    return t.view(torch.uint8 if t.dtype is F8 else torch.int32 if t.dtype is torch.float32 else torch.int16)


def left_alone(buf, view, used, fill):
    """Everything but the used rows is as it was (and ends as it was)."""
    raw(view)[:used] = int(torch.tensor(float(fill)).view(torch.int32)) if view.dtype is torch.float32 else fill
    assert (buf == fill).all()


def parts(rows, width, per_value):
    """Ranges of rows that are small calls."""
    step = max(1, (STREAM // 2) // (per_value * width))
    return [slice(a, min(a + step, rows)) for a in range(0, rows, step)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("gated,out,group", [(True, True, None), (True, False, 128), (True, True, 32), (False, False, 64),
                                             (False, True, 128)])
def test_act(name, width, gated, out, group):
    dt = TYPES[name]
    g = torch.Generator(device=DEV).manual_seed(width)
    rows = rows_of(width, 4)
    wide = width * (2 if gated else 1)
    _, x = place(rows, wide, dt, 5, 3, 0)
    x.copy_(normal(g, rows, wide, dt=dt))
    if gated:
        x[::97, 1] = -95.0                                       # (another way to the sigmoid)
    for used in used_of(rows, width):
        at = torch.tensor([0, used // 3, used], dtype=torch.int32, device=DEV) if used < rows else None
        outs = {}
        if out:
            outs["out"] = place(rows, width, dt, 3, 1, 77)
        if group:
            outs["out8"] = place(rows, width, F8, 1, 2, 77)
            outs["scales"] = place(rows, -(-width // group), torch.float32, 2, 1, 77)
        hr.experts_act(x, gated=gated, offsets=at, group=group or 128, **{n: v for n, (_, v) in outs.items()})
        want = {n: torch.empty(used, v.shape[1], dtype=v.dtype, device=DEV) for n, (_, v) in outs.items()}
        for rs in parts(used, width, 4):
            hr.experts_act(x[rs], gated=gated, group=group or 128, **{n: v[rs] for n, v in want.items()})
        for n, (buf, view) in outs.items():
            assert torch.equal(raw(view)[:used], raw(want[n])), n
            left_alone(buf, view, used, 77)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("again,same", [(False, False), (True, False), (True, True)])
def test_act_grad(name, width, again, same):
    dt = TYPES[name]
    g = torch.Generator(device=DEV).manual_seed(width + 1)
    rows = rows_of(width, 10)
    values = normal(g, rows, 2 * width, dt=dt)
    values[::97, 1] = -95.0
    _, dy = place(rows, width, dt, 1, 1, 0)
    dy.copy_(normal(g, rows, width, dt=dt))
    for used in used_of(rows, width):
        at = torch.tensor([0, used // 3, used], dtype=torch.int32, device=DEV) if used < rows else None
        dx_buf, dx = place(rows, 2 * width, dt, 3, 1, 77)
        out_buf, out = place(rows, width, dt, 1, 2, 77)
        x = values
        if same:
            dx.copy_(values)
            x = dx
        hr.experts_act_grad(dy, x, dx, out=out if again else None, offsets=at)
        want, want_out = (torch.empty(used, w, dtype=dt, device=DEV) for w in (2 * width, width))
        for rs in parts(used, width, 10):
            hr.experts_act_grad(dy[rs], values[rs], want[rs], out=want_out[rs])
        assert torch.equal(raw(dx)[:used], raw(want))
        if same:
            assert torch.equal(raw(dx)[used:], raw(values)[used:])
            raw(dx)[used:] = 77
        left_alone(dx_buf, dx, used, 77)
        if again:
            assert torch.equal(raw(out)[:used], raw(want_out))
        left_alone(out_buf, out, used if again else 0, 77)


def test_captured():
    """Large calls in a graph, replayed with fresh values beside eager small ones."""
    g = torch.Generator(device=DEV).manual_seed(5)
    width, dt = 2056, torch.bfloat16
    rows = rows_of(width, 4)
    x, dy = (torch.empty(rows, w, dtype=dt, device=DEV) for w in (2 * width, width))
    out, again, dx = (torch.empty(rows, w, dtype=dt, device=DEV) for w in (width, width, 2 * width))
    codes, scales = torch.empty(rows, width, dtype=F8, device=DEV), torch.empty(rows, -(-width // 128), device=DEV)

    def calls():
        hr.experts_act(x, out, out8=codes, scales=scales)
        hr.experts_act_grad(dy, x, dx, out=again)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        x.copy_(normal(g, rows, 2 * width, dt=dt))
        dy.copy_(normal(g, rows, width, dt=dt))
        for t in (out, again, dx, codes, scales):
            raw(t).zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = [torch.empty_like(t) for t in (out, codes, scales, dx)]
        for rs in parts(rows, width, 10):
            hr.experts_act(x[rs], want[0][rs], out8=want[1][rs], scales=want[2][rs])
            hr.experts_act_grad(dy[rs], x[rs], want[3][rs])
        for a, b in zip((out, codes, scales, dx, again), (*want, want[0])):
            assert torch.equal(raw(a), raw(b))
