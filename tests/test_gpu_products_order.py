"""GPU: which calls of the experts' products give equal bits, and which only equal
sums within the roundings of two orders."""
import pytest
import torch

from _gpu import needs_gpu
from _products import F8, grad_ref, product_ref, sum_tol, wide_blocks, wide_rows
from _rows import Maker, within
from message_fp16_all_amd import hr

pytestmark = [pytest.mark.gpu, needs_gpu]
DEV = "cuda:0"
EXPERTS = 3
SPLIT = [0, 2, 2, 5]                                             # fifths of the rows

# (rows, k, n): a few rows, whose waves split k; ordinary ones; large tiles
SIZES = [(10, 528, 272), (330, 272, 1040), (6000, 144, 2576)]


def put(values, offset, extra, dt):
    """``values`` (matrices or rows) at a distance from a 16-byte address, rows further apart; NaN around them."""
    lead, width = values.shape[:-1].numel(), values.shape[-1]
    size = 1 if dt is F8 else 2
    buf = torch.full((offset + lead * (width + extra) + 64,), 0x7F if size == 1 else 0x7FFF,
                     dtype=torch.uint8 if size == 1 else torch.int16, device=DEV)
    strides = [width + extra, 1]
    if values.dim() == 3:
        strides.insert(0, values.shape[1] * (width + extra))
    view = buf.as_strided(values.shape, strides, offset)
    view.copy_(values.view(buf.dtype).to(DEV))
    return view.view(dt)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("rows,k,n", SIZES)
def test_product(kind, transposed, rows, k, n):
    m = Maker(rows)
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    offsets = [rows * f // 5 for f in SPLIT]
    shape = (EXPERTS, *((k, n) if transposed else (n, k)))
    scales = {}
    if kind == "e4m3":
        inside = F8
        x, w = (m.normal(*s, sigma=20.0).clamp(-448, 448).to(F8) for s in ((rows, k), shape))
        xs = torch.exp2(m.normal(rows, -(-k // 128)))
        ws = torch.exp2(m.normal(EXPERTS, *(-(-v // 128) for v in shape[1:])) - 8)
        scales = dict(x_scales=xs.to(DEV), w_scales=ws.to(DEV))
        ref, mag = product_ref(wide_rows(x, xs), wide_blocks(w, ws), offsets, transposed)
    else:
        inside = dt
        x, w = m.normal(rows, k, dtype=dt), m.normal(*shape, dtype=dt)
        ref, mag = product_ref(x, w, offsets, transposed)
    unit = 16 // (1 if kind == "e4m3" else 2)
    at = torch.tensor(offsets, dtype=torch.int32, device=DEV)

    def run(x_at, w_at, shift=0):
        out = torch.empty(rows, n + 3, dtype=dt, device=DEV)[:, shift:n + shift]
        hr.experts_product(put(x, *x_at, inside), put(w, *w_at, inside), out, offsets=at, transposed=transposed, **scales)
        return out.contiguous()

    def same(a, b):
        return torch.equal(a.view(torch.int16), b.view(torch.int16))

    whole = run((0, 0), (0, 0))
    assert same(whole, run((0, 0), (0, 0), 1))
    assert same(whole, run((unit, 2 * unit), (3 * unit, unit), 2))
    odd = run((1, 0), (0, 0))
    for x_at, w_at in (((1, 3), (0, 0)), ((0, 0), (unit - 1, 0)), ((5, 0), (2, 1))):
        assert same(odd, run(x_at, w_at))
    tol = sum_tol(dt, ref, mag, k, eight=kind == "e4m3")
    within(whole, ref, tol, "in whole units")
    within(odd, ref, tol, "at odd addresses")


@pytest.mark.parametrize("f32", [False, True])
# rows split over waves; ordinary and large tiles
@pytest.mark.parametrize("rows,k,n", [(400, 136, 72), (200, 1544, 2056), (90, 2056, 4104)])
def test_gradient(f32, rows, k, n):
    m, dt = Maker(rows + 1), torch.float16
    offsets = [rows * f // 5 for f in SPLIT]
    dy, x = m.normal(rows, n, dtype=dt), m.normal(rows, k, dtype=dt)
    to = torch.float32 if f32 else dt
    at = torch.tensor(offsets, dtype=torch.int32, device=DEV)

    def run(dy_at, x_at):
        dw = torch.empty(EXPERTS, n, k, dtype=to, device=DEV)
        hr.experts_product_grad(put(dy, *dy_at, dt), put(x, *x_at, dt), dw, offsets=at)
        return dw

    whole = run((0, 0), (0, 0))
    assert torch.equal(whole, run((8, 16), (24, 8)))
    odd = run((1, 0), (0, 0))
    assert torch.equal(odd, run((0, 1), (3, 0))) and torch.equal(odd, run((0, 0), (0, 5)))
    ref, mag = grad_ref(dy, x, offsets)
    tol = sum_tol(to, ref, mag, rows)
    within(whole, ref, tol, "in whole units")
    within(odd, ref, tol, "at odd addresses")
